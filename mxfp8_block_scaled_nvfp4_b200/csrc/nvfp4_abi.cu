// libnvfp4.so: the C ABI of include/nvfp4.h.  Host-side argument checks
// (texts after ops.cpp validate_global_scale / validate_qqmm_inputs,
// "mlx 0.30.7.2 -> 0.30.7.6" diff, page 8), launch configuration and the
// device error word.  One translation unit: the kernels live in the .cuh
// files it includes.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "nvfp4.h"
#include "common.cuh"
#include "quantize.cuh"
#include "qmv.cuh"
#include "qmv_tc.cuh"
#include "qqmm_sm100.cuh"
#include "gather_qmm.cuh"
#include "kv_cache.cuh"
#include "kv_append.cuh"
#include "kv_attention.cuh"
#include "kv_prefill.cuh"
#include "norm.cuh"

using namespace nvfp4;

// Scratch of gather_qmm_noalloc: a fixed device array that the library owns
// for the life of the process (1 MiB on every GPU that loads the library).
// Host code must not pass the symbol itself to a kernel -- on the host it
// only names the array; the device address comes from
// cudaGetSymbolAddress, looked up once per device (see noalloc_scratch).
static constexpr size_t kNoAllocScratchBytes = (size_t)1 << 20;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

namespace {

thread_local char t_msg[512] = "";

nvfp4_status fail(nvfp4_status s, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(t_msg, sizeof(t_msg), fmt, ap);
  va_end(ap);
  return s;
}

nvfp4_status ok() {
  t_msg[0] = '\0';
  return NVFP4_OK;
}

nvfp4_status check_launch(const char* what) {
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[%s] launch failed: %s", what, cudaGetErrorString(e));
  return ok();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// a * b > limit for a, b >= 0, without forming the (possibly overflowing) product.
bool product_exceeds(int64_t a, int64_t b, int64_t limit) { return b != 0 && a > limit / b; }

struct DeviceInfo {
  int sm_count = 0;
  int cc_major = 0;
  int cc_minor = 0;
  bool ok = false;
};

DeviceInfo g_dev[64];
std::mutex g_dev_mu;

// Current device's properties; the library runs on sm_100 (B200) only.
nvfp4_status device_info(const char* tag, DeviceInfo* out) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[%s] cudaGetDevice: %s", tag, cudaGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] device ordinal %d", tag, dev);
  std::lock_guard<std::mutex> lk(g_dev_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ok) {
    if (cudaDeviceGetAttribute(&d.sm_count, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.cc_major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.cc_minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess)
      return fail(NVFP4_ERR_CUDA, "[%s] cudaDeviceGetAttribute failed", tag);
    d.ok = true;
  }
  if (d.cc_major != 10 || d.cc_minor != 0)
    return fail(NVFP4_ERR_UNSUPPORTED,
                "[%s] this library is built for sm_100a (B200); device has compute capability %d.%d",
                tag, d.cc_major, d.cc_minor);
  *out = d;
  return NVFP4_OK;
}

int64_t dt_size(nvfp4_dtype dt) { return dt == NVFP4_DT_F32 ? 4 : 2; }

bool valid_dt(nvfp4_dtype dt) { return dt == NVFP4_DT_F32 || dt == NVFP4_DT_F16 || dt == NVFP4_DT_BF16; }

// CTAs of `fn` (threads per CTA, dynamic shared memory) that fit on one SM
// at once, cached per kernel and CTA size.
int resident_ctas(const void* fn, int threads, size_t smem) {
  struct Known {
    const void* fn;
    int threads, ctas;
  };
  static std::mutex mu;
  static Known known[512];
  static int n = 0;
  std::lock_guard<std::mutex> lk(mu);
  for (int i = 0; i < n; ++i)
    if (known[i].fn == fn && known[i].threads == threads) return known[i].ctas;
  int b = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, fn, threads, smem) != cudaSuccess || b < 1) b = 1;
  if (n < 512) known[n++] = Known{fn, threads, b};
  return b;
}

// Persistent elementwise grid: every SM filled with as many CTAs of the
// kernel as are resident at once (one wave), never more than the work needs.
unsigned ew_grid(const DeviceInfo& d, uint64_t work_threads, int per_sm) {
  uint64_t want = (work_threads + kEwThreads - 1) / kEwThreads;
  uint64_t cap = (uint64_t)d.sm_count * (uint64_t)per_sm;
  if (want > cap) want = cap;
  if (want < 1) want = 1;
  return (unsigned)want;
}

template <typename F>
void dispatch_dt(nvfp4_dtype dt, F&& f) {
  switch (dt) {
    case NVFP4_DT_F32: f(float{}); break;
    case NVFP4_DT_F16: f(__half{}); break;
    default: f(__nv_bfloat16{}); break;
  }
}

template <typename F>
void dispatch_mode(nvfp4_mode mode, F&& f) {
  switch (mode) {
    case NVFP4_MODE_NVFP4: f(std::integral_constant<int, kv::kNV>{}); break;
    case NVFP4_MODE_MXFP8: f(std::integral_constant<int, kv::kMX8>{}); break;
    default: f(std::integral_constant<int, kv::kMX4>{}); break;
  }
}

constexpr int64_t kMaxElems = (int64_t)1 << 34;  // 16 Gi elements: 32-bit half-block indices

// How a norm kernel lays a row of `blocks` 16-element blocks over a CTA: one
// block a thread where the rows are 32-byte aligned and fit (K <= 8192), else
// four; row_warps warps a row, `warps` a CTA (as many rows as make about eight).
struct NormPlan {
  bool one;
  uint32_t row_warps, warps;
};
NormPlan norm_plan(int64_t blocks, bool aligned) {
  NormPlan p;
  p.one = aligned && blocks <= norm::kMaxThreads;
  const int64_t per_warp = p.one ? 32 : 128;
  p.row_warps = (uint32_t)((blocks + per_warp - 1) / per_warp);
  p.warps = p.row_warps >= 8 ? p.row_warps : 8 / p.row_warps * p.row_warps;
  return p;
}
template <typename F>
void dispatch_norm(const NormPlan& p, F&& f) {
  if (p.one) f(std::integral_constant<int, 1>{});
  else f(std::integral_constant<int, 4>{});
}
bool aligned32(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 31u) == 0; }

}  // namespace

extern "C" {

const char* nvfp4_status_string(nvfp4_status s) {
  switch (s) {
    case NVFP4_OK: return "ok";
    case NVFP4_ERR_INVALID_ARG: return "invalid argument";
    case NVFP4_ERR_UNSUPPORTED: return "unsupported";
    case NVFP4_ERR_CUDA: return "CUDA error";
    case NVFP4_ERR_TIMEOUT: return "device wait timed out";
    case NVFP4_ERR_DEVICE_INDEX: return "device-side index out of range";
  }
  return "unknown status";
}

const char* nvfp4_last_error_message(void) { return t_msg; }

nvfp4_status nvfp4_check_device_errors(nvfp4_stream_t stream) {
  cudaError_t e = cudaStreamSynchronize(stream);
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[check_device_errors] %s", cudaGetErrorString(e));
  unsigned int word = 0;
  e = cudaMemcpyFromSymbol(&word, g_device_error, sizeof(word));
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[check_device_errors] %s", cudaGetErrorString(e));
  if (word != 0) {
    const unsigned int zero = 0;
    cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
    if (word & kDevErrTimeout)
      return fail(NVFP4_ERR_TIMEOUT, "[device] a kernel gave up a bounded wait (word 0x%x)", word);
    return fail(NVFP4_ERR_DEVICE_INDEX, "[device] an index was out of range (word 0x%x)", word);
  }
  return ok();
}

size_t nvfp4_scale_bytes(int64_t rows, int64_t cols, nvfp4_layout layout) {
  if (rows < 0 || cols < 0) return 0;
  if (layout == NVFP4_LAYOUT_LINEAR) return (size_t)(rows * cols);
  return (size_t)(((rows + 127) / 128 * 128) * ((cols + 3) / 4 * 4));
}

static nvfp4_status amax_launch(const char* tag, const nvfp4_amax_item* items, int count, nvfp4_dtype dt,
                                nvfp4_stream_t stream) {
  if (!valid_dt(dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] dtype must be float32, float16 or bfloat16", tag);
  if (!items || count < 1 || count > kAmaxSegs)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] between 1 and %d tensors, got %d", tag, kAmaxSegs, count);
  for (int i = 0; i < count; ++i) {
    const nvfp4_amax_item& it = items[i];
    if (it.n < 0 || it.n > kMaxElems) return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad size %lld", tag, (long long)it.n);
    if (!it.g_out || (it.n > 0 && !it.x)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
    if (!aligned16(it.x) || (reinterpret_cast<uintptr_t>(it.g_out) & 3u))
      return fail(NVFP4_ERR_INVALID_ARG, "[%s] x must be 16-byte aligned, g_out 4-byte aligned", tag);
    for (int j = 0; j < i; ++j)
      if (items[j].g_out == it.g_out) return fail(NVFP4_ERR_INVALID_ARG, "[%s] two tensors share one output", tag);
  }
  DeviceInfo d;
  nvfp4_status st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  // outputs start at 0 (max |x| >= 0); one memset when they are consecutive floats
  bool consecutive = true;
  for (int i = 1; i < count; ++i) consecutive = consecutive && items[i].g_out == items[0].g_out + i;
  cudaError_t e = cudaSuccess;
  if (consecutive) {
    e = cudaMemsetAsync(items[0].g_out, 0, sizeof(float) * (size_t)count, stream);
  } else {
    for (int i = 0; i < count && e == cudaSuccess; ++i) e = cudaMemsetAsync(items[i].g_out, 0, sizeof(float), stream);
  }
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[%s] memset: %s", tag, cudaGetErrorString(e));
  AmaxSegs a;
  memset(&a, 0, sizeof(a));
  uint64_t vecs = 0;
  for (int i = 0; i < count; ++i) {
    if (items[i].n == 0) continue;  // its output stays 0
    a.x[a.count] = items[i].x;
    a.n[a.count] = items[i].n;
    a.out[a.count] = items[i].g_out;
    ++a.count;
    vecs += (uint64_t)(items[i].n / 8 + 1);
  }
  if (a.count == 0) return ok();
  dispatch_dt(dt, [&](auto tag_t) {
    using T = decltype(tag_t);
    const unsigned grid = ew_grid(d, (vecs + 3) / 4, resident_ctas((const void*)k_amax<T>, kEwThreads, 0));
    k_amax<T><<<grid, kEwThreads, 0, stream>>>(a);
  });
  return check_launch(tag);
}

nvfp4_status nvfp4_amax(const void* x, nvfp4_dtype dt, int64_t n, float* g_out, nvfp4_stream_t stream) {
  const nvfp4_amax_item it{x, n, g_out};
  return amax_launch("amax", &it, 1, dt, stream);
}

nvfp4_status nvfp4_amax_multi(const nvfp4_amax_item* items, int count, nvfp4_dtype dt, nvfp4_stream_t stream) {
  return amax_launch("amax_multi", items, count, dt, stream);
}

// Argument checks of one row-wise quantize; *empty is set when the output
// has no element.  kind: 0 NVFP4, 1 MXFP8, 2 MXFP4 (the two MX kinds use
// 32-element blocks).
static nvfp4_status check_quantize(const char* tag, int kind, const void* x, nvfp4_dtype dt, int64_t rows,
                                   int64_t K, const float* g, const uint32_t* codes, const uint8_t* scales,
                                   nvfp4_layout layout, bool* empty) {
  const int group = kind ? 32 : 16;
  if (!valid_dt(dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] dtype must be float32, float16 or bfloat16", tag);
  if (layout != NVFP4_LAYOUT_LINEAR && layout != NVFP4_LAYOUT_SWIZZLED)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] unknown scale layout", tag);
  if (rows < 0 || K < 0 || product_exceeds(rows, K, kMaxElems))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad shape [%lld, %lld]", tag, (long long)rows, (long long)K);
  if (K % group != 0)
    return fail(NVFP4_ERR_INVALID_ARG,
                "[%s] The last dimension of the matrix needs to be divisible by the quantization group size %d. "
                "However the provided matrix has shape [%lld, %lld]",
                tag, group, (long long)rows, (long long)K);
  if (rows * K > 0 && (!x || !codes || !scales)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || (reinterpret_cast<uintptr_t>(g) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned", tag);
  *empty = rows * K == 0;
  return NVFP4_OK;
}

static ScaleOut scale_out(uint8_t* scales, int64_t K, int group, nvfp4_layout layout) {
  ScaleOut so;
  so.init(scales, (uint32_t)(K / group), layout == NVFP4_LAYOUT_SWIZZLED);
  return so;
}

// NVFP4 quantize of `count` tensors (those with elements) in one launch.
static nvfp4_status nvfp4_quantize_launch(const char* tag, const nvfp4_quantize_item* items, int count,
                                          nvfp4_dtype dt, nvfp4_stream_t stream, bool sr, uint64_t seed) {
  if (!items || count < 1 || count > kMaxSegs)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] between 1 and %d tensors, got %d", tag, kMaxSegs, count);
  QuantSegs q;
  memset(&q, 0, sizeof(q));
  q.seed = seed;
  bool v8 = true;  // 256-bit loads need every input 32-byte aligned
  for (int i = 0; i < count; ++i) {
    const nvfp4_quantize_item& it = items[i];
    bool empty = false;
    nvfp4_status st = check_quantize(tag, 0, it.x, dt, it.rows, it.K, it.g, it.codes, it.scales, it.layout, &empty);
    if (st != NVFP4_OK) return st;
    if (empty) continue;
    QuantSeg& sg = q.s[q.count++];
    sg.x = it.x;
    sg.g = it.g;
    sg.codes = it.codes;
    sg.so = scale_out(it.scales, it.K, 16, it.layout);
    sg.rows = (uint32_t)it.rows;
    sg.n_blk = (uint32_t)(it.rows * it.K / 16);
    sg.first_unit = q.units;
    q.units += (sg.n_blk + kUnitBlk - 1) / kUnitBlk;
    v8 = v8 && (reinterpret_cast<uintptr_t>(it.x) & 31u) == 0;
  }
  if (q.count == 0) return ok();  // nothing to write: no device work, no device query
  DeviceInfo d;
  nvfp4_status st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  dispatch_dt(dt, [&](auto tag_t) {
    using T = decltype(tag_t);
    auto go = [&](auto kern) {
      const unsigned grid = ew_grid(d, (uint64_t)q.units * 32u, resident_ctas((const void*)kern, kEwThreads, 0));
      kern<<<grid, kEwThreads, 0, stream>>>(q);
    };
    if (sr) v8 ? go(k_nvfp4_quantize<T, true, true>) : go(k_nvfp4_quantize<T, true, false>);
    else v8 ? go(k_nvfp4_quantize<T, false, true>) : go(k_nvfp4_quantize<T, false, false>);
  });
  return check_launch(tag);
}

static nvfp4_status mx_quantize(const char* tag, int kind, const void* x, nvfp4_dtype dt, int64_t rows, int64_t K,
                                uint32_t* codes, uint8_t* scales, nvfp4_layout layout, nvfp4_stream_t stream) {
  bool empty = false;
  nvfp4_status st = check_quantize(tag, kind, x, dt, rows, K, nullptr, codes, scales, layout, &empty);
  if (st != NVFP4_OK) return st;
  if (empty) return ok();  // nothing to write: no device work, no device query
  DeviceInfo d;
  st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  const ScaleOut so = scale_out(scales, K, 32, layout);
  const uint32_t n_half = (uint32_t)(rows * K / 8);
  dispatch_dt(dt, [&](auto tag_t) {
    using T = decltype(tag_t);
    const void* fn = kind == 1 ? (const void*)k_mxfp8_quantize<T> : (const void*)k_mxfp4_quantize<T>;
    const unsigned grid = ew_grid(d, ((uint64_t)n_half + kUnroll - 1) / kUnroll, resident_ctas(fn, kEwThreads, 0));
    if (kind == 1)
      k_mxfp8_quantize<T><<<grid, kEwThreads, 0, stream>>>(static_cast<const T*>(x), n_half, codes, so,
                                                           (uint32_t)rows);
    else
      k_mxfp4_quantize<T><<<grid, kEwThreads, 0, stream>>>(static_cast<const T*>(x), n_half, codes, so,
                                                           (uint32_t)rows);
  });
  return check_launch(tag);
}

nvfp4_status nvfp4_quantize(const void* x, nvfp4_dtype dt, int64_t rows, int64_t K, const float* g,
                            uint32_t* codes, uint8_t* scales, nvfp4_layout layout, nvfp4_stream_t stream) {
  const nvfp4_quantize_item it{x, rows, K, g, codes, scales, layout};
  return nvfp4_quantize_launch("quantize", &it, 1, dt, stream, false, 0);
}

nvfp4_status nvfp4_quantize_multi(const nvfp4_quantize_item* items, int count, nvfp4_dtype dt,
                                  nvfp4_stream_t stream) {
  return nvfp4_quantize_launch("quantize_multi", items, count, dt, stream, false, 0);
}

nvfp4_status nvfp4_quantize_sr(const void* x, nvfp4_dtype dt, int64_t rows, int64_t K, const float* g,
                               uint64_t seed, uint32_t* codes, uint8_t* scales, nvfp4_layout layout,
                               nvfp4_stream_t stream) {
  const nvfp4_quantize_item it{x, rows, K, g, codes, scales, layout};
  return nvfp4_quantize_launch("quantize_sr", &it, 1, dt, stream, true, seed);
}

static nvfp4_status columnwise_launch(const char* tag, const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols,
                                      const float* g, uint32_t* codes, uint8_t* scales, nvfp4_layout layout,
                                      nvfp4_stream_t stream, bool sr, uint64_t seed) {
  if (!valid_dt(dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] dtype must be float32, float16 or bfloat16", tag);
  if (layout != NVFP4_LAYOUT_LINEAR && layout != NVFP4_LAYOUT_SWIZZLED)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] unknown scale layout", tag);
  if (rows < 0 || cols < 0 || rows > (1 << 30) || cols > (1 << 30) || rows * cols > kMaxElems)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad shape [%lld, %lld]", tag, (long long)rows, (long long)cols);
  if (rows % 16 != 0)
    return fail(NVFP4_ERR_INVALID_ARG,
                "[%s] The quantized dimension (rows of x, the last dimension of x^T) needs to be divisible by the "
                "quantization group size 16. However the provided matrix has shape [%lld, %lld]",
                tag, (long long)rows, (long long)cols);
  if (rows * cols > 0 && (!x || !codes || !scales)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (!aligned16(x) || !aligned16(codes) || !aligned16(scales) || (reinterpret_cast<uintptr_t>(g) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned", tag);
  if (rows * cols == 0) return ok();
  DeviceInfo d;
  nvfp4_status st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  ScaleOut so;
  so.init(scales, (uint32_t)(rows / 16), layout == NVFP4_LAYOUT_SWIZZLED);
  dim3 grid((unsigned)((rows + kColR - 1) / kColR), (unsigned)((cols + kColC - 1) / kColC));
  dispatch_dt(dt, [&](auto tag_t) {
    using T = decltype(tag_t);
    if (sr)
      k_nvfp4_quantize_columnwise<T, true><<<grid, kColThreads, 0, stream>>>(static_cast<const T*>(x), (uint32_t)rows,
                                                                            (uint32_t)cols, g, codes, so, seed);
    else
      k_nvfp4_quantize_columnwise<T><<<grid, kColThreads, 0, stream>>>(static_cast<const T*>(x), (uint32_t)rows,
                                                                        (uint32_t)cols, g, codes, so);
  });
  return check_launch(tag);
}

nvfp4_status nvfp4_quantize_columnwise(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, const float* g,
                                       uint32_t* codes, uint8_t* scales, nvfp4_layout layout, nvfp4_stream_t stream) {
  return columnwise_launch("quantize_columnwise", x, dt, rows, cols, g, codes, scales, layout, stream, false, 0);
}

nvfp4_status nvfp4_quantize_columnwise_sr(const void* x, nvfp4_dtype dt, int64_t rows, int64_t cols, const float* g,
                                          uint64_t seed, uint32_t* codes, uint8_t* scales, nvfp4_layout layout,
                                          nvfp4_stream_t stream) {
  return columnwise_launch("quantize_columnwise_sr", x, dt, rows, cols, g, codes, scales, layout, stream, true, seed);
}

nvfp4_status mxfp8_quantize(const void* x, nvfp4_dtype dt, int64_t rows, int64_t K, uint32_t* codes,
                            uint8_t* scales, nvfp4_layout layout, nvfp4_stream_t stream) {
  return mx_quantize("mxfp8_quantize", 1, x, dt, rows, K, codes, scales, layout, stream);
}

nvfp4_status mxfp4_quantize(const void* x, nvfp4_dtype dt, int64_t rows, int64_t K, uint32_t* codes,
                            uint8_t* scales, nvfp4_layout layout, nvfp4_stream_t stream) {
  return mx_quantize("mxfp4_quantize", 2, x, dt, rows, K, codes, scales, layout, stream);
}

static nvfp4_status dequantize_common(const char* tag, int kind, const uint32_t* codes, const uint8_t* scales,
                                      nvfp4_layout layout, int64_t rows, int64_t K, const float* g, void* out,
                                      nvfp4_dtype out_dt, nvfp4_stream_t stream) {
  const int group = kind ? 32 : 16;
  if (!valid_dt(out_dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] output dtype must be float32, float16 or bfloat16", tag);
  if (layout != NVFP4_LAYOUT_LINEAR && layout != NVFP4_LAYOUT_SWIZZLED)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] unknown scale layout", tag);
  if (rows < 0 || K < 0 || product_exceeds(rows, K, kMaxElems) || K % group != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad shape [%lld, %lld] for group size %d", tag, (long long)rows,
                (long long)K, group);
  if (rows * K > 0 && (!codes || !scales || !out)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (!aligned16(codes) || !aligned16(scales) || !aligned16(out) || (reinterpret_cast<uintptr_t>(g) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned", tag);
  if (rows * K == 0) return ok();  // nothing to write: no device work, no device query
  DeviceInfo d;
  nvfp4_status st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  ScaleIn si;
  si.p = scales;
  si.blocks_per_row = (uint32_t)(K / group);
  si.Cp = (uint32_t)((K / group + 3) / 4 * 4);
  si.swizzled = layout == NVFP4_LAYOUT_SWIZZLED;
  const uint32_t n_half = (uint32_t)(rows * K / 8);
  dispatch_dt(out_dt, [&](auto tag_t) {
    using T = decltype(tag_t);
    const void* fn = kind == 1 ? (const void*)k_mxfp8_dequantize<T>
                     : kind == 2 ? (const void*)k_mxfp4_dequantize<T> : (const void*)k_nvfp4_dequantize<T>;
    const unsigned grid = ew_grid(d, n_half, resident_ctas(fn, kEwThreads, 0));
    if (kind == 1)
      k_mxfp8_dequantize<T><<<grid, kEwThreads, 0, stream>>>(codes, si, n_half, static_cast<T*>(out));
    else if (kind == 2)
      k_mxfp4_dequantize<T><<<grid, kEwThreads, 0, stream>>>(codes, si, n_half, static_cast<T*>(out));
    else
      k_nvfp4_dequantize<T><<<grid, kEwThreads, 0, stream>>>(codes, si, g, n_half, static_cast<T*>(out));
  });
  return check_launch(tag);
}

nvfp4_status nvfp4_dequantize(const uint32_t* codes, const uint8_t* scales, nvfp4_layout layout, int64_t rows,
                              int64_t K, const float* g, void* out, nvfp4_dtype out_dt, nvfp4_stream_t stream) {
  return dequantize_common("dequantize", 0, codes, scales, layout, rows, K, g, out, out_dt, stream);
}

nvfp4_status mxfp8_dequantize(const uint32_t* codes, const uint8_t* scales, nvfp4_layout layout, int64_t rows,
                              int64_t K, void* out, nvfp4_dtype out_dt, nvfp4_stream_t stream) {
  return dequantize_common("mxfp8_dequantize", 1, codes, scales, layout, rows, K, nullptr, out, out_dt, stream);
}

nvfp4_status mxfp4_dequantize(const uint32_t* codes, const uint8_t* scales, nvfp4_layout layout, int64_t rows,
                              int64_t K, void* out, nvfp4_dtype out_dt, nvfp4_stream_t stream) {
  return dequantize_common("mxfp4_dequantize", 2, codes, scales, layout, rows, K, nullptr, out, out_dt, stream);
}

nvfp4_status nvfp4_swizzle_scales(const uint8_t* lin, int64_t rows, int64_t cols, uint8_t* swz,
                                  nvfp4_stream_t stream) {
  if (rows < 0 || cols < 0 || product_exceeds(rows, cols, (int64_t)1 << 31))
    return fail(NVFP4_ERR_INVALID_ARG, "[swizzle_scales] bad shape");
  if (rows * cols > 0 && (!lin || !swz)) return fail(NVFP4_ERR_INVALID_ARG, "[swizzle_scales] null pointer");
  if (!aligned16(lin) || !aligned16(swz))
    return fail(NVFP4_ERR_INVALID_ARG, "[swizzle_scales] Starting addresses must be 16-byte aligned");
  if (rows * cols == 0) return ok();
  DeviceInfo d;
  nvfp4_status st = device_info("swizzle_scales", &d);
  if (st != NVFP4_OK) return st;
  const uint32_t Rp = (uint32_t)((rows + 127) / 128 * 128), Cp = (uint32_t)((cols + 3) / 4 * 4);
  const unsigned grid = ew_grid(d, (uint64_t)Rp * Cp, resident_ctas((const void*)k_swizzle_scales, kEwThreads, 0));
  k_swizzle_scales<<<grid, kEwThreads, 0, stream>>>(lin, (uint32_t)rows, (uint32_t)cols, Rp, Cp, swz);
  return check_launch("swizzle_scales");
}

// Global-scale checks of qqmm ("mlx 0.30.7.2 -> 0.30.7.6" diff, page 8,
// ops.cpp validate_global_scale and validate_qqmm_inputs).
static nvfp4_status check_qqmm_global_scales(nvfp4_mode mode, const float* g_x, const float* g_w) {
  if (mode != NVFP4_MODE_NVFP4 && (g_x || g_w))
    return fail(NVFP4_ERR_INVALID_ARG, "[qqmm] Global scale is only supported for 'nvfp4' quantization mode.");
  if (mode == NVFP4_MODE_NVFP4 && ((g_x == nullptr) != (g_w == nullptr)))
    return fail(NVFP4_ERR_INVALID_ARG,
                "[qqmm] For nvfp4 mode, either both global_scale_x and global_scale_w must be provided, or neither.");
  return NVFP4_OK;
}

nvfp4_status qqmm(nvfp4_mode mode, int64_t M, int64_t N, int64_t K, const uint32_t* a_codes,
                  const uint8_t* a_scales, const uint32_t* b_codes, const uint8_t* b_scales, const float* g_x,
                  const float* g_w, void* y, nvfp4_dtype y_dt, nvfp4_stream_t stream) {
  if (mode != NVFP4_MODE_NVFP4 && mode != NVFP4_MODE_MXFP8 && mode != NVFP4_MODE_MXFP4)
    return fail(NVFP4_ERR_INVALID_ARG, "[qqmm] Only 'nvfp4', 'mxfp8' and 'mxfp4' modes are supported.");
  nvfp4_status st = check_qqmm_global_scales(mode, g_x, g_w);
  if (st != NVFP4_OK) return st;
  if (!valid_dt(y_dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[qqmm] output dtype must be float32, float16 or bfloat16");
  if (M < 0 || N < 0 || K < 0 || M > (1 << 30) || N > (1 << 30) || K > (1 << 30))
    return fail(NVFP4_ERR_INVALID_ARG, "[qqmm] bad shape");
  if (K % 32 != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "[qqmm] K must be a multiple of 32, got %lld", (long long)K);
  if (K == 0 && M * N > 0) return fail(NVFP4_ERR_INVALID_ARG, "[qqmm] K must be positive when M*N > 0");
  if (M * N > 0 && (!a_codes || !a_scales || !b_codes || !b_scales || !y))
    return fail(NVFP4_ERR_INVALID_ARG, "[qqmm] null pointer");
  if (!aligned16(a_codes) || !aligned16(b_codes) || !aligned16(a_scales) || !aligned16(b_scales) || !aligned16(y) ||
      (reinterpret_cast<uintptr_t>(g_x) & 3u) || (reinterpret_cast<uintptr_t>(g_w) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[qqmm] tensor pointers must be 16-byte aligned");
  if (M * N == 0) return ok();
  DeviceInfo d;
  st = device_info("qqmm", &d);
  if (st != NVFP4_OK) return st;
  return qqmm_launch((int)mode, M, N, K, a_codes, a_scales, b_codes, b_scales, g_x, g_w, y,
                     (int)y_dt, d.sm_count, stream, t_msg, sizeof(t_msg));
}

// pdl: the tensor-core kernel's PDL form (qmv_pdl); the SIMT kernel always
// launches in plain stream order.
static nvfp4_status qmv_launch(const void* x, nvfp4_dtype x_dt, const float* g_x, const uint32_t* w_codes,
                               const uint8_t* w_scales, const float* g_w, int64_t M, int64_t N, int64_t K, void* y,
                               nvfp4_stream_t stream, bool pdl) {
  if (!valid_dt(x_dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[qmv] dtype must be float32, float16 or bfloat16");
  if ((g_x == nullptr) != (g_w == nullptr))
    return fail(NVFP4_ERR_INVALID_ARG,
                "[qqmm] For nvfp4 mode, either both global_scale_x and global_scale_w must be provided, or neither.");
  if (M < 1 || M > kQmvMaxM) return fail(NVFP4_ERR_INVALID_ARG, "[qmv] M must be in [1, %d], got %lld", kQmvMaxM, (long long)M);
  if (N < 0 || K < 32 || K % 32 != 0 || N > (1 << 30))
    return fail(NVFP4_ERR_INVALID_ARG, "[qmv] bad shape N=%lld K=%lld (K %% 32 == 0)", (long long)N, (long long)K);
  if (M * K * 4 > 160 * 1024)
    return fail(NVFP4_ERR_UNSUPPORTED, "[qmv] M*K*4 bytes of x_hat must fit 160 KiB of shared memory");
  if (N > 0 && (!x || !w_codes || !w_scales || !y)) return fail(NVFP4_ERR_INVALID_ARG, "[qmv] null pointer");
  if (!aligned16(x) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) ||
      (reinterpret_cast<uintptr_t>(g_x) & 3u) || (reinterpret_cast<uintptr_t>(g_w) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[qmv] tensor pointers must be 16-byte aligned");
  if (N == 0) return ok();
  DeviceInfo d;
  nvfp4_status st = device_info("qmv", &d);
  if (st != NVFP4_OK) return st;
  cudaError_t e = cudaSuccess;
  const uint32_t esz = x_dt == NVFP4_DT_F32 ? 4u : 2u;
  const uint32_t stages = qtc::pick_stages(M, K, esz);
  if (stages > 0) {
    // tensor-core path: one CTA per 128 weight rows
    CUtensorMap mw;
    if (!qtc::make_map(&mw, w_codes, (uint64_t)N, (uint64_t)K))
      return fail(NVFP4_ERR_CUDA, "[qmv] cuTensorMapEncodeTiled failed");
    const qtc::Groups gr = qtc::pick_groups(stages, (uint32_t)(K / 256));
    qtc::Args a{x, g_x, w_codes, w_scales, g_w, y, (uint32_t)M, (uint32_t)N, (uint32_t)K, stages, gr.g0, gr.g};
    const uint32_t MM = M == 1 ? 1u : 2u;
    const size_t smem = qtc::smem_needed(stages, MM, (uint32_t)K, esz);
    const unsigned grid = (unsigned)((N + qtc::BM - 1) / qtc::BM);
    dispatch_dt(x_dt, [&](auto tag_t) {
      using T = decltype(tag_t);
      auto go = [&](auto kern) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return;
        if (!pdl) {
          kern<<<grid, qtc::THREADS, smem, stream>>>(mw, a);
          return;
        }
        cudaLaunchConfig_t cfg;
        memset(&cfg, 0, sizeof(cfg));
        cfg.gridDim = dim3(grid);
        cfg.blockDim = dim3(qtc::THREADS);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kern, mw, a);
      };
      if (M == 1) pdl ? go(qtc::k_qmv_tc<T, 1, true>) : go(qtc::k_qmv_tc<T, 1>);
      else pdl ? go(qtc::k_qmv_tc<T, 2, true>) : go(qtc::k_qmv_tc<T, 2>);
    });
  } else {
    const size_t smem = (size_t)M * K * sizeof(float);
    // one CTA of 16 warps per SM; each warp owns whole weight rows
    uint64_t grid = ((uint64_t)N + (kQmvThreads / 32) - 1) / (kQmvThreads / 32);
    if (grid > (uint64_t)d.sm_count) grid = d.sm_count;
    dispatch_dt(x_dt, [&](auto tag_t) {
      using T = decltype(tag_t);
      auto x_t = [](const void* p) { return static_cast<const T*>(p); };
      auto y_t = [](void* p) { return static_cast<T*>(p); };
      auto go = [&](auto kern) {
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e == cudaSuccess)
          kern<<<(unsigned)grid, kQmvThreads, smem, stream>>>(x_t(x), g_x, w_codes, w_scales, g_w, (int)M, (int)N,
                                                             (int)K, y_t(y));
      };
      if (M == 1) go(k_qmv<T, 1>);
      else if (M == 2) go(k_qmv<T, 2>);
      else if (M <= 4) go(k_qmv<T, 4>);
      else go(k_qmv<T, 8>);
    });
  }
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[qmv] %s", cudaGetErrorString(e));
  return check_launch("qmv");
}

nvfp4_status qmv(const void* x, nvfp4_dtype x_dt, const float* g_x, const uint32_t* w_codes, const uint8_t* w_scales,
                 const float* g_w, int64_t M, int64_t N, int64_t K, void* y, nvfp4_stream_t stream) {
  return qmv_launch(x, x_dt, g_x, w_codes, w_scales, g_w, M, N, K, y, stream, false);
}

nvfp4_status qmv_mx(nvfp4_mode mode, const void* x, nvfp4_dtype x_dt, const uint32_t* w_codes,
                    const uint8_t* w_scales, int64_t M, int64_t N, int64_t K, void* y, nvfp4_stream_t stream) {
  if (mode != NVFP4_MODE_MXFP8 && mode != NVFP4_MODE_MXFP4)
    return fail(NVFP4_ERR_INVALID_ARG, "[qmv_mx] mode must be mxfp8 or mxfp4 (nvfp4: use qmv)");
  if (!valid_dt(x_dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[qmv_mx] dtype must be float32, float16 or bfloat16");
  if (M < 1 || M > kQmvMaxM)
    return fail(NVFP4_ERR_INVALID_ARG, "[qmv_mx] M must be in [1, %d], got %lld", kQmvMaxM, (long long)M);
  if (N < 0 || K < 32 || K % 32 != 0 || N > (1 << 30))
    return fail(NVFP4_ERR_INVALID_ARG, "[qmv_mx] bad shape N=%lld K=%lld (K %% 32 == 0)", (long long)N, (long long)K);
  if (M * K * 4 > 160 * 1024)
    return fail(NVFP4_ERR_UNSUPPORTED, "[qmv_mx] M*K*4 bytes of x_hat must fit 160 KiB of shared memory");
  if (N > 0 && (!x || !w_codes || !w_scales || !y)) return fail(NVFP4_ERR_INVALID_ARG, "[qmv_mx] null pointer");
  if (!aligned16(x) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y))
    return fail(NVFP4_ERR_INVALID_ARG, "[qmv_mx] tensor pointers must be 16-byte aligned");
  if (N == 0) return ok();
  DeviceInfo d;
  nvfp4_status st = device_info("qmv_mx", &d);
  if (st != NVFP4_OK) return st;
  const size_t smem = (size_t)M * K * sizeof(float);
  uint64_t grid = ((uint64_t)N + (kQmvThreads / 32) - 1) / (kQmvThreads / 32);
  if (grid > (uint64_t)d.sm_count) grid = d.sm_count;
  cudaError_t e = cudaSuccess;
  dispatch_dt(x_dt, [&](auto tag_t) {
    using T = decltype(tag_t);
    auto go = [&](auto kern) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (e == cudaSuccess)
        kern<<<(unsigned)grid, kQmvThreads, smem, stream>>>(static_cast<const T*>(x), w_codes, w_scales, (int)M,
                                                            (int)N, (int)K, static_cast<T*>(y));
    };
    auto pick = [&](auto mode_tag) {
      constexpr int MD = decltype(mode_tag)::value;
      if (M == 1) go(k_qmv_mx<T, MD, 1>);
      else if (M == 2) go(k_qmv_mx<T, MD, 2>);
      else if (M <= 4) go(k_qmv_mx<T, MD, 4>);
      else go(k_qmv_mx<T, MD, 8>);
    };
    if (mode == NVFP4_MODE_MXFP8) pick(std::integral_constant<int, 1>{});
    else pick(std::integral_constant<int, 2>{});
  });
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[qmv_mx] %s", cudaGetErrorString(e));
  return check_launch("qmv_mx");
}

nvfp4_status qmv_pdl(const void* x, nvfp4_dtype x_dt, const float* g_x, const uint32_t* w_codes,
                     const uint8_t* w_scales, const float* g_w, int64_t M, int64_t N, int64_t K, void* y,
                     nvfp4_stream_t stream) {
  return qmv_launch(x, x_dt, g_x, w_codes, w_scales, g_w, M, N, K, y, stream, true);
}

size_t gather_qmm_workspace_size(int64_t T, int64_t topk, int64_t E) {
  if (T < 0 || topk < 1 || E < 1 || E > gq::MAX_E || product_exceeds(T, topk, 1 << 30)) return 0;
  return gather_workspace_bytes(T, topk, E);
}

size_t gather_qmm_staged_workspace_size(int64_t T, int64_t topk, int64_t E, int64_t K) {
  if (T < 0 || topk < 1 || E < 1 || E > gq::MAX_E || K < 0 || K > (1 << 30) || product_exceeds(T, topk, 1 << 30))
    return 0;
  const int64_t P = T * topk;
  if (K > 0 && P > (int64_t)(SIZE_MAX / 4) / K) return 0;
  return gather_staged_workspace_bytes(T, topk, E, K);
}

// Host checks shared by the gather entries: shapes (K % 64, N % n_mult, K > 0
// when there is output), pointers and, where the caller passes one
// (check_ws), the workspace size.
static nvfp4_status check_gather(const char* tag, bool kn, const void* x, const uint32_t* w_codes,
                                 const uint8_t* w_scales, const float* g, const int32_t* idx, int64_t T,
                                 int64_t topk, int64_t E, int64_t N, int64_t K, const void* y, bool check_ws,
                                 const void* workspace, size_t workspace_bytes) {
  if (T < 0 || topk < 1 || E < 1 || N < 0 || K < 0 || product_exceeds(T, topk, 1 << 30) || N > (1 << 30) ||
      K > (1 << 30))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad shape", tag);
  const int n_mult = kn ? 32 : 16;
  if (K % 64 != 0 || N % n_mult != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] K must be a multiple of 64 and N of %d (K=%lld N=%lld)", tag, n_mult,
                (long long)K, (long long)N);
  if (K == 0 && T * N > 0) return fail(NVFP4_ERR_INVALID_ARG, "[%s] K must be positive when T*N > 0", tag);
  if (E > gq::MAX_E) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] at most %d experts, got %lld", tag, gq::MAX_E, (long long)E);
  // The weight tensor map has E*N rows ([E, N, K]) or E*K rows ([E, K, N]);
  // TMA row coordinates are 32-bit signed.
  const int64_t w_rows = E * (kn ? K : N);
  if (w_rows > INT32_MAX)
    return fail(NVFP4_ERR_UNSUPPORTED, "[%s] the weights span %lld rows; at most %d", tag, (long long)w_rows,
                INT32_MAX);
  if (check_ws && workspace_bytes < gather_workspace_bytes(T, topk, E))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] workspace too small: %zu < %zu", tag, workspace_bytes,
                gather_workspace_bytes(T, topk, E));
  if (T * N > 0 && (!x || !w_codes || !w_scales || !idx || !y || (check_ws && !workspace)))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (!aligned16(x) || !aligned16(w_codes) || !aligned16(w_scales) || !aligned16(y) || !aligned16(workspace) ||
      !aligned16(idx) || !aligned16(g))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned", tag);
  return NVFP4_OK;
}

nvfp4_status gather_qmm(const void* x, const uint32_t* w_codes, const uint8_t* w_scales, const float* g,
                        const int32_t* idx, int64_t T, int64_t topk, int64_t E, int64_t N, int64_t K, void* y,
                        void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  nvfp4_status st = check_gather("gather_qmm", false, x, w_codes, w_scales, g, idx, T, topk, E, N, K, y, true,
                                 workspace, workspace_bytes);
  if (st != NVFP4_OK) return st;
  if (T * N == 0) return ok();
  DeviceInfo d;
  st = device_info("gather_qmm", &d);
  if (st != NVFP4_OK) return st;
  return gather_qmm_launch(x, w_codes, w_scales, g, idx, T, topk, E, N, K, y, workspace, workspace_bytes, d.sm_count,
                           stream, t_msg, sizeof(t_msg));
}

nvfp4_status gather_qmm_kn(const void* x, const uint32_t* w_codes, const uint8_t* w_scales, const float* g,
                        const int32_t* idx, int64_t T, int64_t topk, int64_t E, int64_t N, int64_t K, void* y,
                        void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  nvfp4_status st = check_gather("gather_qmm_kn", true, x, w_codes, w_scales, g, idx, T, topk, E, N, K, y, true,
                                 workspace, workspace_bytes);
  if (st != NVFP4_OK) return st;
  if (T * N == 0) return ok();
  DeviceInfo d;
  st = device_info("gather_qmm_kn", &d);
  if (st != NVFP4_OK) return st;
  return gather_qmm_launch(x, w_codes, w_scales, g, idx, T, topk, E, N, K, y, workspace, workspace_bytes, d.sm_count,
                           stream, t_msg, sizeof(t_msg), true);
}

// Identity of the calling thread's current context (0 if none can be read):
// cuCtxGetCurrent and cuCtxGetId through the runtime's driver entry points,
// so the library needs no link against the driver library.
static unsigned long long current_context_id() {
  using GetCurrent = CUresult (*)(CUcontext*);
  using GetId = CUresult (*)(CUcontext, unsigned long long*);
  static GetCurrent get_current = nullptr;
  static GetId get_id = nullptr;
  static bool looked = false;
  if (!looked) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_current = reinterpret_cast<GetCurrent>(p);
    if (cudaGetDriverEntryPoint("cuCtxGetId", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<GetId>(p);
    looked = true;
  }
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (!get_current || !get_id || get_current(&ctx) != CUDA_SUCCESS || !ctx || get_id(ctx, &id) != CUDA_SUCCESS)
    return 0;
  return id;
}

// Device address of g_noalloc_scratch on the current device, resolved with
// that device current and cached per device together with the context it
// belongs to: a new context on the device (after cudaDeviceReset, which
// unloads the library's module and may place the array elsewhere) resolves
// it again.
static nvfp4_status noalloc_scratch(void** out) {
  static void* addr[64] = {nullptr};
  static unsigned long long ctx_of[64] = {0};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[gather_qmm_noalloc] cudaGetDevice: %s", cudaGetErrorString(e));
  if (dev < 0 || dev >= 64) return fail(NVFP4_ERR_UNSUPPORTED, "[gather_qmm_noalloc] device ordinal %d", dev);
  std::lock_guard<std::mutex> lk(mu);
  const unsigned long long ctx = current_context_id();
  if (addr[dev] == nullptr || ctx == 0 || ctx != ctx_of[dev]) {
    void* p = nullptr;
    e = cudaGetSymbolAddress(&p, g_noalloc_scratch);
    if (e != cudaSuccess || p == nullptr)
      return fail(NVFP4_ERR_CUDA, "[gather_qmm_noalloc] cudaGetSymbolAddress of the static scratch failed: %s",
                  cudaGetErrorString(e));
    addr[dev] = p;
    ctx_of[dev] = ctx;
  }
  *out = addr[dev];
  return NVFP4_OK;
}

nvfp4_status gather_qmm_noalloc(const void* x, const uint32_t* w_codes, const uint8_t* w_scales, const float* g,
                                const int32_t* idx, int64_t T, int64_t topk, int64_t E, int64_t N, int64_t K,
                                void* y, nvfp4_stream_t stream) {
  nvfp4_status st = check_gather("gather_qmm_noalloc", false, x, w_codes, w_scales, g, idx, T, topk, E, N, K, y,
                                 false, nullptr, 0);
  if (st != NVFP4_OK) return st;
  if (T * N == 0) return ok();
  const size_t need = gather_workspace_bytes(T, topk, E);
  if (need > kNoAllocScratchBytes)
    return fail(NVFP4_ERR_UNSUPPORTED,
                "[gather_qmm_noalloc] T=%lld, topk=%lld, E=%lld needs %zu bytes of scratch; the static scratch "
                "holds %zu bytes (use gather_qmm with a caller-provided workspace)",
                (long long)T, (long long)topk, (long long)E, need, kNoAllocScratchBytes);
  void* scratch = nullptr;
  st = noalloc_scratch(&scratch);
  if (st != NVFP4_OK) return st;
  // The routing kernel rewrites every scratch entry the grouped kernel reads
  // (tile count, tile list, permutation; the staging kernel the staged rows
  // of every routed pair), so nothing needs clearing between calls.
  return gather_qmm(x, w_codes, w_scales, g, idx, T, topk, E, N, K, y, scratch, kNoAllocScratchBytes, stream);
}

// ---------------------------------------------------------------------------
// Root-mean-square norm
// ---------------------------------------------------------------------------
constexpr int64_t kNormMaxK = 32768;

static nvfp4_status check_norm(const char* tag, nvfp4_dtype dt, int64_t rows, int64_t K, int64_t group) {
  if (!valid_dt(dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] dtype must be float32, float16 or bfloat16", tag);
  if (rows < 0 || K < 0 || product_exceeds(rows, K, kMaxElems))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad shape [%lld, %lld]", tag, (long long)rows, (long long)K);
  if (K < group || K % group != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] K must be a positive multiple of %lld, got %lld", tag, (long long)group, (long long)K);
  if (K > kNormMaxK)
    return fail(NVFP4_ERR_UNSUPPORTED, "[%s] K must be at most %lld, got %lld", tag, (long long)kNormMaxK, (long long)K);
  return NVFP4_OK;
}

// mode: nvfp4_mode or norm::kPlain.
static nvfp4_status rms_norm_launch(const char* tag, int mode, const void* x, const void* residual, const void* w,
                                    nvfp4_dtype dt, int64_t rows, int64_t K, double eps, const float* g, void* h,
                                    void* y, uint8_t* scales, nvfp4_layout layout, float* rstd, nvfp4_stream_t stream) {
  const int64_t group = mode == kv::kMX8 || mode == kv::kMX4 ? 32 : 16;
  nvfp4_status st = check_norm(tag, dt, rows, K, group);
  if (st != NVFP4_OK) return st;
  if (layout != NVFP4_LAYOUT_LINEAR && layout != NVFP4_LAYOUT_SWIZZLED)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] unknown scale layout", tag);
  if (g && mode != kv::kNV) return fail(NVFP4_ERR_INVALID_ARG, "[%s] Global scales are only supported for 'nvfp4' mode.", tag);
  if (!(eps >= 0x1p-126 && eps <= 0x1p126))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] eps must be in [2^-126, 2^126], got %g", tag, eps);
  if (rows > 0 && (!x || !w || !y || (mode != norm::kPlain && !scales))) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (rows > 0 && (residual == nullptr) != (h == nullptr))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] h must be given with a residual, and only then", tag);
  if (!aligned16(x) || !aligned16(residual) || !aligned16(w) || !aligned16(h) || !aligned16(y) || !aligned16(scales) ||
      (reinterpret_cast<uintptr_t>(g) & 3u) || (reinterpret_cast<uintptr_t>(rstd) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned (g and rstd 4-byte)", tag);
  if (rows == 0) return ok();
  DeviceInfo d;
  st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  norm::Args a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.residual = residual;
  a.w = w;
  a.h = h;
  a.y = y;
  a.rstd = rstd;
  a.g = g;
  if (mode != norm::kPlain) a.so = scale_out(scales, K, (int)group, layout);
  a.rows = rows;
  a.K = (uint32_t)K;
  a.blocks = (uint32_t)(K / 16);
  a.eps = eps;
  a.per_k = 1.0 / (double)K;
  const bool v8 = aligned32(x) && aligned32(residual) && aligned32(w) && aligned32(h) && (mode != norm::kPlain || aligned32(y)) &&
                  K * dt_size(dt) % 32 == 0;
  const NormPlan p = norm_plan(a.blocks, v8);
  a.row_warps = p.row_warps;
  const int64_t rpc = p.warps / p.row_warps, want = (rows + rpc - 1) / rpc;
  dispatch_dt(dt, [&](auto tag_t) {
    using T = decltype(tag_t);
    dispatch_norm(p, [&](auto u) {
      constexpr int U = decltype(u)::value;
      auto go = [&](auto kern) {
        const int64_t cap = (int64_t)d.sm_count * resident_ctas((const void*)kern, (int)p.warps * 32, 0);
        kern<<<(unsigned)(want < cap ? want : cap), p.warps * 32u, 0, stream>>>(a);
      };
      if (mode == kv::kNV) go(norm::k_rms_norm<T, kv::kNV, U>);
      else if (mode == kv::kMX8) go(norm::k_rms_norm<T, kv::kMX8, U>);
      else if (mode == kv::kMX4) go(norm::k_rms_norm<T, kv::kMX4, U>);
      else go(norm::k_rms_norm<T, norm::kPlain, U>);
    });
  });
  return check_launch(tag);
}

nvfp4_status rms_norm(const void* x, const void* residual, const void* w, nvfp4_dtype dt, int64_t rows, int64_t K,
                      double eps, void* h, void* y, float* rstd, nvfp4_stream_t stream) {
  return rms_norm_launch("rms_norm", norm::kPlain, x, residual, w, dt, rows, K, eps, nullptr, h, y, nullptr,
                         NVFP4_LAYOUT_LINEAR, rstd, stream);
}

nvfp4_status rms_norm_quantize(nvfp4_mode mode, const void* x, const void* residual, const void* w, nvfp4_dtype dt,
                               int64_t rows, int64_t K, double eps, const float* g, void* h, uint32_t* codes,
                               uint8_t* scales, nvfp4_layout layout, float* rstd, nvfp4_stream_t stream) {
  const char* tag = "rms_norm_quantize";
  if (mode != NVFP4_MODE_NVFP4 && mode != NVFP4_MODE_MXFP8 && mode != NVFP4_MODE_MXFP4)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] mode must be 'nvfp4', 'mxfp8' or 'mxfp4'", tag);
  return rms_norm_launch(tag, mode, x, residual, w, dt, rows, K, eps, g, h, codes, scales, layout, rstd, stream);
}

// CTAs of k_rms_norm_vjp, each with a part of dw.
static int64_t norm_vjp_ctas(const NormPlan& p, int64_t rows) {
  const int64_t rpc = p.warps / p.row_warps, want = (rows + rpc - 1) / rpc, most = p.warps > 8 ? 148 : 148 * 2;
  return want < most ? want : most;
}

size_t rms_norm_vjp_workspace_size(int64_t rows, int64_t K) {
  if (rows < 1 || K < 16 || K % 16 != 0 || K > kNormMaxK || product_exceeds(rows, K, kMaxElems)) return 0;
  const NormPlan p = norm_plan(K / 16, true);
  return (size_t)norm_vjp_ctas(p, rows) * (size_t)K * 4;
}

nvfp4_status rms_norm_vjp(const void* dy, const void* h, const void* w, const float* rstd, const void* dh,
                          nvfp4_dtype dt, int64_t rows, int64_t K, void* dx, float* dw, void* workspace,
                          size_t workspace_bytes, nvfp4_stream_t stream) {
  const char* tag = "rms_norm_vjp";
  nvfp4_status st = check_norm(tag, dt, rows, K, 16);
  if (st != NVFP4_OK) return st;
  if (rows > 0 && (!dy || !h || !w || !rstd || !dx)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (!aligned16(dy) || !aligned16(h) || !aligned16(w) || !aligned16(dh) || !aligned16(dx) || !aligned16(dw) ||
      !aligned16(workspace) || (reinterpret_cast<uintptr_t>(rstd) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned (rstd 4-byte)", tag);
  if (dw && (workspace_bytes < rms_norm_vjp_workspace_size(rows, K) || (rows > 0 && !workspace)))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] dw needs a workspace of %zu bytes, got %zu", tag,
                rms_norm_vjp_workspace_size(rows, K), workspace_bytes);
  if (rows == 0 && !dw) return ok();
  DeviceInfo d;
  st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  norm::VjpArgs a;
  memset(&a, 0, sizeof(a));
  a.dy = dy;
  a.h = h;
  a.w = w;
  a.rstd = rstd;
  a.dh = dh;
  a.dx = dx;
  a.dw = dw;
  a.part = static_cast<float*>(workspace);
  a.rows = rows;
  a.K = (uint32_t)K;
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    const NormPlan p = norm_plan(K / 16, true);
    a.row_warps = p.row_warps;
    const int64_t ctas = norm_vjp_ctas(p, rows);
    a.parts = (uint32_t)ctas;
    dispatch_dt(dt, [&](auto tag_t) {
      using T = decltype(tag_t);
      if (!p.one) {
        norm::k_rms_norm_vjp<T, false><<<(unsigned)ctas, p.warps * 32u, 0, stream>>>(a);
        return;
      }
      auto kern = norm::k_rms_norm_vjp<T, true>;
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(norm::kMaxThreads * norm::kVjpSmem<T>));
      if (e == cudaSuccess) kern<<<(unsigned)ctas, p.warps * 32u, p.warps * 32u * norm::kVjpSmem<T>, stream>>>(a);
    });
  }
  if (dw && e == cudaSuccess) {  // its launch overlaps the kernel before it
    cudaLaunchConfig_t cfg;
    memset(&cfg, 0, sizeof(cfg));
    cfg.gridDim = dim3((unsigned)((K + 31) / 32));
    cfg.blockDim = dim3(norm::kDwThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = rows > 0 ? 1 : 0;
    e = cudaLaunchKernelEx(&cfg, norm::k_rms_norm_dw, a);
  }
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[%s] %s", tag, cudaGetErrorString(e));
  return check_launch(tag);
}

// Checks of a cache handle that every cache call makes.
static nvfp4_status check_kv_cache(const char* tag, const nvfp4_kv_cache* c) {
  if (!c) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null cache", tag);
  if (c->mode != NVFP4_MODE_NVFP4 && c->mode != NVFP4_MODE_MXFP8 && c->mode != NVFP4_MODE_MXFP4)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] mode must be 'nvfp4', 'mxfp8' or 'mxfp4'", tag);
  if (c->mode != NVFP4_MODE_NVFP4 && (c->g_k || c->g_v))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] Global scales are only supported for 'nvfp4' mode.", tag);
  if ((c->g_k == nullptr) != (c->g_v == nullptr))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] either both g_k and g_v must be provided, or neither.", tag);
  if (c->num_pages < 0 || c->page_size < 1 || product_exceeds(c->num_pages, c->page_size, INT32_MAX) ||
      c->page_size > INT32_MAX)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad cache of %lld pages of %lld rows (fewer than 2^31 rows in all)", tag,
                (long long)c->num_pages, (long long)c->page_size);
  if (c->heads < 1 || c->heads > 65535)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] heads must be in [1, 65535], got %lld", tag, (long long)c->heads);
  if (c->D < 32 || c->D % 32 != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] D must be a positive multiple of 32, got %lld", tag, (long long)c->D);
  if (c->D > 256) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] D must be at most 256, got %lld", tag, (long long)c->D);
  if (c->num_pages > 0 && (!c->k_codes || !c->k_scales || !c->v_codes || !c->v_scales))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] null cache pointer", tag);
  if (!aligned16(c->k_codes) || !aligned16(c->k_scales) || !aligned16(c->v_codes) || !aligned16(c->v_scales) ||
      (reinterpret_cast<uintptr_t>(c->g_k) & 3u) || (reinterpret_cast<uintptr_t>(c->g_v) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned", tag);
  return NVFP4_OK;
}

// Token stride of a [T, width] operand whose rows may be parts of longer ones.
static bool bad_stride(int64_t T, int64_t stride, int64_t width, nvfp4_dtype dt) {
  return T > 1 && (stride < width || stride > INT32_MAX || stride * dt_size(dt) % 16 != 0);
}

// Every row (of a multiple of 32 elements) begins at a multiple of 32 bytes.
static bool rows_aligned32(const void* p, int64_t T, int64_t stride, nvfp4_dtype dt) {
  return (reinterpret_cast<uintptr_t>(p) & 31u) == 0 && (T <= 1 || stride * dt_size(dt) % 32 == 0);
}

static kv::RowArgs kv_row_args(const nvfp4_kv_cache* c, int64_t T, const int32_t* slots) {
  kv::RowArgs a;
  memset(&a, 0, sizeof(a));
  a.codes[0] = reinterpret_cast<uint8_t*>(c->k_codes);
  a.codes[1] = reinterpret_cast<uint8_t*>(c->v_codes);
  a.scales[0] = c->k_scales;
  a.scales[1] = c->v_scales;
  a.g[0] = c->g_k;
  a.g[1] = c->g_v;
  a.slots = slots;
  a.T = (uint32_t)T;
  a.heads = (uint32_t)c->heads;
  a.D = (uint32_t)c->D;
  a.page_size = (uint32_t)c->page_size;
  a.num_slots = (uint32_t)(c->num_pages * c->page_size);
  a.units = (uint32_t)(T * c->heads * c->D / 16);
  a.per_head.init(a.D / 16u);
  a.per_token.init(a.heads * (a.D / 16u));
  a.by_page.init(a.page_size);
  return a;
}

nvfp4_status kv_cache_write(const nvfp4_kv_cache* cache, const void* k, const void* v, nvfp4_dtype dt, int64_t T,
                            int64_t k_stride, int64_t v_stride, const int32_t* slots, nvfp4_stream_t stream) {
  const char* tag = "kv_cache_write";
  nvfp4_status st = check_kv_cache(tag, cache);
  if (st != NVFP4_OK) return st;
  if (!valid_dt(dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] dtype must be float32, float16 or bfloat16", tag);
  const int64_t width = cache->heads * cache->D;
  if (T < 0 || product_exceeds(T, width, kMaxElems)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad T=%lld", tag, (long long)T);
  if (bad_stride(T, k_stride, width, dt) || bad_stride(T, v_stride, width, dt))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] token strides must be at least heads*D and a multiple of 16 bytes", tag);
  if (T > 0 && (!k || !v || !slots)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slots) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned (slots 4-byte)", tag);
  if (T == 0) return ok();
  DeviceInfo d;
  st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  kv::RowArgs a = kv_row_args(cache, T, slots);
  a.x[0] = k;
  a.x[1] = v;
  a.stride[0] = k_stride;
  a.stride[1] = v_stride;
  const bool v8 = rows_aligned32(k, T, k_stride, dt) && rows_aligned32(v, T, v_stride, dt);
  const dim3 grid((a.units + kv::kRowThreads - 1) / kv::kRowThreads, 2);
  dispatch_dt(dt, [&](auto tag_t) {
    using E = decltype(tag_t);
    dispatch_mode(cache->mode, [&](auto m) {
      constexpr int MODE = decltype(m)::value;
      if (v8) kv::k_kv_write<E, MODE, true><<<grid, kv::kRowThreads, 0, stream>>>(a);
      else kv::k_kv_write<E, MODE, false><<<grid, kv::kRowThreads, 0, stream>>>(a);
    });
  });
  return check_launch(tag);
}

nvfp4_status kv_cache_read(const nvfp4_kv_cache* cache, const int32_t* slots, int64_t T, void* k_out, void* v_out,
                           nvfp4_dtype out_dt, nvfp4_stream_t stream) {
  const char* tag = "kv_cache_read";
  nvfp4_status st = check_kv_cache(tag, cache);
  if (st != NVFP4_OK) return st;
  if (!valid_dt(out_dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] dtype must be float32, float16 or bfloat16", tag);
  const int64_t width = cache->heads * cache->D;
  if (T < 0 || product_exceeds(T, width, kMaxElems)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad T=%lld", tag, (long long)T);
  if (T > 0 && (!k_out || !v_out || !slots)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (!aligned16(k_out) || !aligned16(v_out) || (reinterpret_cast<uintptr_t>(slots) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned (slots 4-byte)", tag);
  if (T == 0) return ok();
  DeviceInfo d;
  st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  kv::RowArgs a = kv_row_args(cache, T, slots);
  a.x[0] = k_out;
  a.x[1] = v_out;
  a.stride[0] = a.stride[1] = width;
  const bool v8 = rows_aligned32(k_out, T, width, out_dt) && rows_aligned32(v_out, T, width, out_dt);
  const dim3 grid((a.units + kv::kRowThreads - 1) / kv::kRowThreads, 2);
  dispatch_dt(out_dt, [&](auto tag_t) {
    using E = decltype(tag_t);
    dispatch_mode(cache->mode, [&](auto m) {
      constexpr int MODE = decltype(m)::value;
      if (v8) kv::k_kv_read<E, MODE, true><<<grid, kv::kRowThreads, 0, stream>>>(a);
      else kv::k_kv_read<E, MODE, false><<<grid, kv::kRowThreads, 0, stream>>>(a);
    });
  });
  return check_launch(tag);
}

nvfp4_status kv_cache_append(const nvfp4_kv_cache* cache, const void* q, const void* k, const void* v, nvfp4_dtype dt,
                             int64_t T, int64_t Hq, int64_t q_stride, int64_t k_stride, int64_t v_stride,
                             const float* cos, const float* sin, int64_t max_pos, int64_t rot, int interleaved,
                             const int32_t* positions, const int32_t* slots, void* q_out, nvfp4_stream_t stream) {
  const char* tag = "kv_cache_append";
  nvfp4_status st = check_kv_cache(tag, cache);
  if (st != NVFP4_OK) return st;
  if (!valid_dt(dt)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] dtype must be float32, float16 or bfloat16", tag);
  if (Hq < 1 || Hq > 65535) return fail(NVFP4_ERR_INVALID_ARG, "[%s] Hq must be in [1, 65535], got %lld", tag, (long long)Hq);
  const int64_t width = cache->heads * cache->D, q_width = Hq * cache->D;
  if (T < 0 || product_exceeds(T, width, kMaxElems) || product_exceeds(T, q_width, kMaxElems))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad T=%lld", tag, (long long)T);
  if (rot < 16 || rot > cache->D || rot % 16 != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] rot must be a multiple of 16 in [16, D], got %lld", tag, (long long)rot);
  if (max_pos < 0 || max_pos > INT32_MAX) return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad max_pos=%lld", tag, (long long)max_pos);
  if (bad_stride(T, q_stride, q_width, dt) || bad_stride(T, k_stride, width, dt) || bad_stride(T, v_stride, width, dt))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] token strides must be at least a token's elements and a multiple of 16 bytes", tag);
  if (T > 0 && (!q || !k || !v || !positions || !slots || !q_out || (max_pos > 0 && (!cos || !sin))))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(cos) || !aligned16(sin) || !aligned16(q_out) ||
      (reinterpret_cast<uintptr_t>(positions) & 3u) || (reinterpret_cast<uintptr_t>(slots) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] tensor pointers must be 16-byte aligned (positions and slots 4-byte)", tag);
  if (T == 0) return ok();
  DeviceInfo d;
  st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  kv::AppendArgs a;
  memset(&a, 0, sizeof(a));
  a.r = kv_row_args(cache, T, slots);
  a.r.x[0] = k;
  a.r.x[1] = v;
  a.r.stride[0] = k_stride;
  a.r.stride[1] = v_stride;
  a.q = q;
  a.q_out = q_out;
  a.q_stride = q_stride;
  a.cs[0] = cos;
  a.cs[1] = sin;
  a.positions = positions;
  a.max_pos = (uint32_t)max_pos;
  a.rot = (uint32_t)rot;
  a.interleaved = interleaved != 0;
  a.Hq = (uint32_t)Hq;
  // four heads a thread from a GPU full of threads with one on (measured at k_kv_append)
  const bool few = T * q_width / 16 < 148 * 2048;
  a.q_groups = few ? a.Hq : (a.Hq + 3) / 4;
  a.q_units = (uint32_t)(T * a.q_groups * (cache->D / 16));
  a.q_per_token.init((uint32_t)(a.q_groups * (cache->D / 16)));
  a.q_ctas = (a.q_units + kv::kRowThreads - 1) / kv::kRowThreads;
  a.kv_ctas = (a.r.units + kv::kRowThreads - 1) / kv::kRowThreads;
  const bool v8 = rows_aligned32(k, T, k_stride, dt) && rows_aligned32(v, T, v_stride, dt);
  dispatch_dt(dt, [&](auto tag_t) {
    using E = decltype(tag_t);
    dispatch_mode(cache->mode, [&](auto m) {
      constexpr int MODE = decltype(m)::value;
      const unsigned grid = a.q_ctas + 2u * a.kv_ctas;
      auto go = [&](auto kern) { kern<<<grid, kv::kRowThreads, 0, stream>>>(a); };
      if (few) v8 ? go(kv::k_kv_append<E, MODE, true, 1>) : go(kv::k_kv_append<E, MODE, false, 1>);
      else v8 ? go(kv::k_kv_append<E, MODE, true, 4>) : go(kv::k_kv_append<E, MODE, false, 4>);
    });
  });
  return check_launch(tag);
}

nvfp4_status kv_cache_move(const nvfp4_kv_cache* cache, const int32_t* src, const int32_t* dst, int64_t M,
                           const int32_t* starts, int64_t S, nvfp4_stream_t stream) {
  const char* tag = "kv_cache_move";
  nvfp4_status st = check_kv_cache(tag, cache);
  if (st != NVFP4_OK) return st;
  if (M < 0 || M > INT32_MAX || S < 0 || S > INT32_MAX || (!starts && S != M))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad M=%lld, S=%lld (without starts, S must equal M)", tag, (long long)M, (long long)S);
  const int64_t blocks = cache->D / (cache->mode == NVFP4_MODE_NVFP4 ? 16 : 32);
  const int64_t code_bytes = cache->D / (cache->mode == NVFP4_MODE_MXFP8 ? 1 : 2);
  const int64_t piece = blocks & -blocks;  // the largest power of two that divides a row's scale bytes: 1 to 16
  const int64_t pieces = code_bytes / 16 + blocks / piece;
  if (product_exceeds(S, cache->heads * 2 * pieces, INT32_MAX))
    return fail(NVFP4_ERR_UNSUPPORTED, "[%s] S*heads*%lld must be below 2^31", tag, (long long)(2 * pieces));
  if (M > 0 && (!src || !dst)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if ((reinterpret_cast<uintptr_t>(src) & 3u) || (reinterpret_cast<uintptr_t>(dst) & 3u) || (reinterpret_cast<uintptr_t>(starts) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] src, dst and starts must be 4-byte aligned", tag);
  if (M == 0 || S == 0) return ok();
  DeviceInfo d;
  st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  kv::MoveArgs a;
  memset(&a, 0, sizeof(a));
  a.codes[0] = reinterpret_cast<uint8_t*>(cache->k_codes);
  a.codes[1] = reinterpret_cast<uint8_t*>(cache->v_codes);
  a.scales[0] = cache->k_scales;
  a.scales[1] = cache->v_scales;
  a.src = src;
  a.dst = dst;
  a.starts = starts;
  a.M = (uint32_t)M;
  a.S = (uint32_t)S;
  a.heads = (uint32_t)cache->heads;
  a.page_size = (uint32_t)cache->page_size;
  a.num_slots = (uint32_t)(cache->num_pages * cache->page_size);
  a.row[0] = (uint32_t)code_bytes;
  a.row[1] = (uint32_t)blocks;
  a.piece = (uint32_t)piece;
  a.code_pieces = (uint32_t)(code_bytes / 16);
  a.pieces = (uint32_t)pieces;
  a.units = (uint32_t)(S * cache->heads * pieces);
  a.per_seq.init((uint32_t)(cache->heads * pieces));
  a.per_head.init((uint32_t)pieces);
  a.by_page.init(a.page_size);
  const unsigned grid = (a.units + kv::kRowThreads - 1) / kv::kRowThreads;
  if (starts) kv::k_kv_move<true><<<grid, kv::kRowThreads, 0, stream>>>(a);
  else kv::k_kv_move<false><<<grid, kv::kRowThreads, 0, stream>>>(a);
  return check_launch(tag);
}

// How kv_attention cuts its work.  k_kv_prefill: rows of queries a CTA holds,
// tokens a CTA walks and the largest number of such chunks a row tile can
// have.  k_kv_decode: rows of a tile; its CTAs share out the rest themselves.
struct KvPlan {
  bool prefill;
  int64_t tile_rows, chunk, chunks;
  size_t bytes_per_chunk;  // k_kv_decode: of partial results per worker
};
constexpr int64_t kKvMaxWorkers = 148 * 4, kKvWorkers = 148;  // most, and fewest worth splitting over
static KvPlan kv_plan(int64_t B, int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t max_q, int64_t max_kv,
                      int64_t window, bool prefill_has_it, bool tree, size_t workspace_bytes) {
  KvPlan p;
  if (max_q > T) max_q = T;
  const int64_t rows = max_q * (Hq / heads);
  // k_kv_decode decodes every code again for each 16 rows (8 above D 128),
  // k_kv_prefill once for 256 (128).  8 heads, group 4, us (k_kv_decode /
  // k_kv_prefill) of 8 sequences of 4096 tokens, and of one of 32768:
  //   D 64, 48 rows   NVFP4 31 / 41, 37 / 39   MXFP4 37 / 46, 45 / 45
  //         64 rows         36 / 42, 44 / 40         45 / 47, 55 / 45
  //   D 128, 32 rows        38 / 50, 43 / 50         52 / 56, 61 / 57
  //          48 rows        49 / 51, 58 / 50         70 / 58, 83 / 57
  //   D 256, 16 rows        54 / 69, 63 / 69         76 / 79, 92 / 79
  //          24 rows        71 / 70, 89 / 70        103 / 80, 131 / 80
  // MXFP8 as MXFP4 (60 / 60, 69 / 60 at D 128 and 32 rows).
  p.prefill = prefill_has_it && rows > (D <= 64 ? 48 : D <= 128 ? 32 : 16);
  p.chunk = p.chunks = 1;
  if (!p.prefill) {
    // D 256: two n-tiles would take more registers than there are.  Trees of at
    // most 8 rows have no variant of their own (24 kernels more): with one, 1 x 2
    // drafts of group 4 over 8192 tokens take 16.4 us for 15.9, 16 of them 46 for
    // 75, and 64 145 for 264 (NVFP4; MXFP4 209 for 417, MXFP8 256 for 469).
    p.tile_rows = (rows <= 8 && !tree) || D > 128 ? 8 : 16;
    p.bytes_per_chunk = (size_t)(2 * p.tile_rows * (D * 4 + 8) + 32);
    return p;
  }
  p.tile_rows = D > 128 ? 128 : 256;
  p.bytes_per_chunk = (size_t)(T * Hq * (D * 4 + 8));
  // tokens a tile's range can span, from a multiple of 16
  int64_t span = max_kv;
  if (window > 0 && window + max_q + 30 < span) span = window + max_q + 30;
  const double tiles = (double)B * (double)heads * (double)((rows + p.tile_rows - 1) / p.tile_rows);
  const double share = (double)span * tiles / 148;  // may exceed 64-bit integers
  int64_t chunk = share < (double)span ? (int64_t)share + 1 : span;
  int64_t fit = workspace_bytes == SIZE_MAX ? span : (int64_t)(workspace_bytes / p.bytes_per_chunk);
  if (fit < 2) fit = 1;
  if (tree) {
    // Few row tiles: as many chunks as take the least time, in tiles of 128
    // tokens: a CTA costs 5 of them besides its own, the join 3.  (144 row tiles
    // over 4160 tokens: 106 us whole, 178 in two chunks.)  That holds for NVFP4,
    // D 128 and two query tiles (2.8 us a tile, 15 a call of one wave besides); a
    // tile is 1.5 to 5.3 us over formats, head sizes and one query tile, and the
    // rest 3 to 6.6 of them.  So flat is the minimum that the choice is within 2 %
    // of the best of 12 numbers of chunks all the same (NVFP4 and MXFP8, D 64, 128
    // and 256, 1 to 12 trees of 32 and 64 drafts over 2048 to 65536 tokens).
    double best = 0;
    for (int64_t c = 1; c <= 64 && c <= fit && (c - 1) * 128 < (span > 0 ? span : 1); ++c) {
      const int64_t each = ((span + c - 1) / c + 127) / 128;
      const double waves = tiles * (double)c / 148, t = (waves > (double)(int64_t)waves ? (int64_t)waves + 1 : (int64_t)waves) * (5.0 + each) + (c > 1 ? 3.0 : 0.0);
      if (c == 1 || t < best) {
        best = t;
        p.chunk = each > 0 ? each * 128 : 128;
      }
    }
    p.chunks = span > 0 ? (span + p.chunk - 1) / p.chunk : 1;
    return p;
  }
  if ((span + fit - 1) / fit > chunk) chunk = (span + fit - 1) / fit;
  p.chunk = (chunk + 127) / 128 * 128;
  if (p.chunk < 512) p.chunk = 512;
  p.chunks = span > 0 ? (span + p.chunk - 1) / p.chunk : 1;
  return p;
}

static size_t kv_workspace(int64_t B, int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t max_q, int64_t max_kv,
                           int64_t window, bool tree) {
  if (B < 1 || B > 65535 || T < 1 || T > (1 << 30) || heads < 1 || heads > 65535 || Hq < 1 || Hq > 65535 ||
      Hq % heads != 0 || D < 32 || D > 256 || D % 32 != 0 || max_q < 1 || max_q > (1 << 30) || max_kv < 0 ||
      max_kv > (1 << 30) || window < 0 || product_exceeds(T, Hq * D, kMaxElems))
    return 0;
  size_t most = 0;  // over the kernels that the types may choose
  for (int i = 0; i < 2; ++i) {
    const KvPlan p = kv_plan(B, T, Hq, heads, D, max_q, max_kv, window > (1 << 30) ? 0 : window, i != 0, tree, SIZE_MAX);
    // 64 tokens are one unit of work: nothing to split
    const size_t bytes = p.prefill ? (p.chunks > 1 ? p.chunks * p.bytes_per_chunk : 0)
                                   : (max_kv > 64 ? (size_t)kKvMaxWorkers * p.bytes_per_chunk : 0);
    if (bytes > most) most = bytes;
  }
  return most;
}

size_t kv_attention_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t max_q,
                                   int64_t max_kv, int64_t window) {
  return kv_workspace(B, T, Hq, heads, D, max_q, max_kv, window, false);
}

size_t kv_attention_tree_workspace_size(int64_t B, int64_t T, int64_t Hq, int64_t heads, int64_t D, int64_t max_q,
                                        int64_t max_kv, int64_t window) {
  return kv_workspace(B, T, Hq, heads, D, max_q, max_kv, window, true);
}

// kv_attention, and with masks over the queries' own tokens kv_attention_tree.
static nvfp4_status kv_attend(const char* tag, const nvfp4_kv_cache* cache, const void* q, nvfp4_dtype q_dt,
                              int64_t q_stride, const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                              int64_t B, int64_t T, int64_t Hq, int64_t max_q, int64_t max_kv, int64_t max_pages,
                              float scale, int causal, int64_t window, const uint32_t* tree, int64_t tree_words, void* out,
                              float* lse, void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  nvfp4_status st = check_kv_cache(tag, cache);
  if (st != NVFP4_OK) return st;
  if (q_dt != NVFP4_DT_F16 && q_dt != NVFP4_DT_BF16)
    return fail(NVFP4_ERR_UNSUPPORTED, "[%s] q must be float16 or bfloat16", tag);
  if (B < 0 || B > 65535 || T < 0 || T > (1 << 30) || Hq < 1 || Hq > 65535 || max_q < 0 || max_q > (1 << 30) ||
      max_pages < 0 || max_pages > INT32_MAX)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] bad sizes B=%lld T=%lld Hq=%lld max_q=%lld max_pages=%lld", tag,
                (long long)B, (long long)T, (long long)Hq, (long long)max_q, (long long)max_pages);
  if (Hq % cache->heads != 0)
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] Hq must be a multiple of the cache's heads, got %lld and %lld", tag,
                (long long)Hq, (long long)cache->heads);
  if (product_exceeds(T, Hq * cache->D, kMaxElems))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] T*Hq*D must be at most 2^34", tag);
  if (max_kv > (1 << 30)) return fail(NVFP4_ERR_UNSUPPORTED, "[%s] max_kv must be at most 2^30", tag);
  if (max_kv < 0 || (max_kv > 0 && (max_pages == 0 || (max_kv - 1) / cache->page_size >= max_pages)))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] max_kv must be in [0, max_pages*page_size], got %lld", tag, (long long)max_kv);
  if (window < 0) return fail(NVFP4_ERR_INVALID_ARG, "[%s] window must not be negative", tag);
  if (!q_start && (T != B || max_q != 1))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] without q_start, T must equal B and max_q be 1", tag);
  if (!(scale - scale == 0.0f)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] scale must be finite", tag);
  if (bad_stride(T, q_stride, Hq * cache->D, q_dt))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] the token stride must be at least Hq*D and a multiple of 16 bytes", tag);
  const bool empty = T == 0 || B == 0 || max_q == 0;
  if (!empty && (!q || !out || !kv_len || (max_pages > 0 && !page_table)))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] null pointer", tag);
  if (workspace_bytes > 0 && !workspace) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null workspace", tag);
  if (!aligned16(q) || !aligned16(out) || !aligned16(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u) ||
      (reinterpret_cast<uintptr_t>(q_start) & 3u) || (reinterpret_cast<uintptr_t>(kv_len) & 3u) ||
      (reinterpret_cast<uintptr_t>(page_table) & 3u))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] q, out and workspace must be 16-byte aligned (lse and the index arrays 4-byte)", tag);
  if (empty) return ok();
  if (max_q > T) max_q = T;  // no sequence has more; the bound sizes the grids
  DeviceInfo d;
  st = device_info(tag, &d);
  if (st != NVFP4_OK) return st;
  kv::AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.codes[0] = reinterpret_cast<const uint8_t*>(cache->k_codes);
  a.codes[1] = reinterpret_cast<const uint8_t*>(cache->v_codes);
  a.scales[0] = cache->k_scales;
  a.scales[1] = cache->v_scales;
  a.g[0] = cache->g_k;
  a.g[1] = cache->g_v;
  a.q = q;
  a.q_stride = T > 1 ? q_stride : Hq * cache->D;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.out = out;
  a.lse = lse;
  a.scale = scale;
  a.B = (uint32_t)B;
  a.T = (uint32_t)T;
  a.Hq = (uint32_t)Hq;
  a.heads = (uint32_t)cache->heads;
  a.G = (uint32_t)(Hq / cache->heads);
  a.D = (uint32_t)cache->D;
  a.max_q = (uint32_t)max_q;
  a.max_kv = (uint32_t)max_kv;
  a.max_pages = (uint32_t)max_pages;
  a.num_pages = (uint32_t)cache->num_pages;
  a.page_size = (uint32_t)cache->page_size;
  a.window = window > (1 << 30) ? 0u : (uint32_t)window;  // a window past any length hides nothing
  a.causal = causal != 0;
  a.tree = tree;
  a.tree_words = (uint32_t)tree_words;
  a.scale_bytes = (uint64_t)cache->num_pages * cache->heads * cache->page_size * (cache->D / (cache->mode == NVFP4_MODE_NVFP4 ? 16 : 32));
  a.by_page.init(a.page_size);
  // k_kv_prefill: no two-term Q for fp16 over the MX modes; it copies some row
  // for every token, so there has to be one
  const bool prefill_has_it = (cache->mode == NVFP4_MODE_NVFP4 || q_dt == NVFP4_DT_BF16) && cache->num_pages > 0;
  const KvPlan p = kv_plan(B, T, Hq, cache->heads, cache->D, max_q, max_kv, a.window, prefill_has_it, tree != nullptr, workspace_bytes);
  a.chunk = (int32_t)p.chunk;
  a.chunks = (uint32_t)p.chunks;
  a.tile_rows = (uint32_t)p.tile_rows;
  const int64_t tiles = (max_q * a.G + p.tile_rows - 1) / p.tile_rows;
  int64_t workers = 0;  // the most that there is workspace for
  if (p.prefill) {
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + (size_t)p.chunks * T * Hq * cache->D * 4);
    if (product_exceeds(tiles, p.chunks, INT32_MAX) || product_exceeds(tiles * p.chunks, B * cache->heads, INT32_MAX))
      return fail(NVFP4_ERR_INVALID_ARG, "[%s] max_q, max_kv and B too large together", tag);
  } else {
    if ((double)B * (double)cache->heads * (double)tiles * ((double)max_kv / 64 + 2) >= 4294967296.0)
      return fail(NVFP4_ERR_UNSUPPORTED, "[%s] B, heads, max_q and max_kv too large together: lower the bounds", tag);
    workers = (int64_t)(workspace_bytes / p.bytes_per_chunk);
    if (workers > kKvMaxWorkers) workers = kKvMaxWorkers;
    a.split = workers >= kKvWorkers && max_kv > 64;
    if (!a.split) workers = kKvMaxWorkers;
    a.part_head = static_cast<int4*>(workspace);
    a.part_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + (size_t)workers * 32);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + (size_t)workers * 2 * p.tile_rows * cache->D);
  }
  cudaError_t e = cudaSuccess;
  dispatch_mode(cache->mode, [&](auto m) {
    constexpr int MODE = decltype(m)::value;
    auto with_type = [&](auto t) {
      using QT = decltype(t);
      // k_kv_decode over row tiles of ROWS
      auto decode = [&](auto kern, auto rows_tag, int smem) {
        constexpr int ROWS = decltype(rows_tag)::value;
        e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return;
        int64_t grid = (int64_t)d.sm_count * resident_ctas((const void*)kern, kv::kDecThreads, (size_t)smem);
        if (grid > workers) grid = workers;
        kern<<<(unsigned)grid, kv::kDecThreads, smem, stream>>>(a);
        if (!a.split) return;
        // the join's launch overlaps the kernel before it
        cudaLaunchConfig_t cfg;
        memset(&cfg, 0, sizeof(cfg));
        cfg.gridDim = dim3((unsigned)grid, ROWS / 2);
        cfg.blockDim = dim3(256);
        cfg.stream = stream;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kv::k_kv_decode_join<QT, ROWS>, a);
      };
      auto with_dim = [&](auto dp) {
        constexpr int DP = decltype(dp)::value;
        if (p.prefill) {
          if constexpr (MODE == kv::kNV || std::is_same<QT, __nv_bfloat16>::value) {
            auto kern = a.tree ? kv::pf::k_kv_prefill<QT, MODE, DP, true> : kv::pf::k_kv_prefill<QT, MODE, DP>;
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kv::pf::Shape<MODE, DP>::smem);
            if (e != cudaSuccess) return;
            kern<<<(unsigned)(tiles * p.chunks * B * cache->heads), kv::pf::THREADS, kv::pf::Shape<MODE, DP>::smem, stream>>>(a);
            if (p.chunks > 1) kv::k_kv_join<QT><<<dim3(a.max_q, a.Hq, a.B), kv::kJoinWarps * 32, 0, stream>>>(a);
          }
          return;
        }
        const bool exact = a.D == (uint32_t)DP;
        constexpr int smem = kv::Geo<MODE, DP>::stages * kv::Geo<MODE, DP>::unit_bytes;
        if constexpr (DP <= 128) {
          if (p.tile_rows == 16) {
            const std::integral_constant<int, 16> r;
            if (a.tree) exact ? decode(kv::k_kv_decode<QT, MODE, DP, 2, true, true>, r, smem) : decode(kv::k_kv_decode<QT, MODE, DP, 2, false, true>, r, smem);
            else exact ? decode(kv::k_kv_decode<QT, MODE, DP, 2, true>, r, smem) : decode(kv::k_kv_decode<QT, MODE, DP, 2, false>, r, smem);
            return;
          }
        }
        const std::integral_constant<int, 8> r;
        if constexpr (DP > 128) {
          if (a.tree) {
            exact ? decode(kv::k_kv_decode<QT, MODE, DP, 1, true, true>, r, smem) : decode(kv::k_kv_decode<QT, MODE, DP, 1, false, true>, r, smem);
            return;
          }
        }
        exact ? decode(kv::k_kv_decode<QT, MODE, DP, 1, true>, r, smem) : decode(kv::k_kv_decode<QT, MODE, DP, 1, false>, r, smem);
      };
      if (a.D <= 64) with_dim(std::integral_constant<int, 64>{});
      else if (a.D <= 128) with_dim(std::integral_constant<int, 128>{});
      else with_dim(std::integral_constant<int, 256>{});
    };
    if (q_dt == NVFP4_DT_F16) with_type(__half{});
    else with_type(__nv_bfloat16{});
  });
  if (e != cudaSuccess) return fail(NVFP4_ERR_CUDA, "[%s] %s", tag, cudaGetErrorString(e));
  return check_launch(tag);
}

nvfp4_status kv_attention(const nvfp4_kv_cache* cache, const void* q, nvfp4_dtype q_dt, int64_t q_stride,
                          const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table, int64_t B,
                          int64_t T, int64_t Hq, int64_t max_q, int64_t max_kv, int64_t max_pages, float scale,
                          int causal, int64_t window, void* out, float* lse, void* workspace, size_t workspace_bytes,
                          nvfp4_stream_t stream) {
  return kv_attend("kv_attention", cache, q, q_dt, q_stride, q_start, kv_len, page_table, B, T, Hq, max_q, max_kv,
                   max_pages, scale, causal, window, nullptr, 0, out, lse, workspace, workspace_bytes, stream);
}

nvfp4_status kv_attention_tree(const nvfp4_kv_cache* cache, const void* q, nvfp4_dtype q_dt, int64_t q_stride,
                               const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                               const uint32_t* tree_mask, int64_t mask_words, int64_t B, int64_t T, int64_t Hq,
                               int64_t max_q, int64_t max_kv, int64_t max_pages, float scale, int64_t window, void* out,
                               float* lse, void* workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  const char* tag = "kv_attention_tree";
  const int64_t most = max_q < T ? max_q : T;
  if (mask_words < 0 || mask_words > (1 << 20) || (most > 0 && (mask_words < 1 || (most - 1) / 32 >= mask_words)))
    return fail(NVFP4_ERR_INVALID_ARG, "[%s] a mask of %lld words does not hold %lld drafts", tag, (long long)mask_words,
                (long long)most);
  if (most > 0 && B > 0 && (!tree_mask || !q_start)) return fail(NVFP4_ERR_INVALID_ARG, "[%s] null tree_mask or q_start", tag);
  if (reinterpret_cast<uintptr_t>(tree_mask) & 3u) return fail(NVFP4_ERR_INVALID_ARG, "[%s] tree_mask must be 4-byte aligned", tag);
  return kv_attend(tag, cache, q, q_dt, q_stride, q_start, kv_len, page_table, B, T, Hq, max_q, max_kv, max_pages, scale, 0,
                   window, tree_mask, mask_words, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
