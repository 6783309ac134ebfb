// k_kv_prefill with masks of drafted tokens as a small library of its own, for
// test_gpu_kv_tree_give_up.py: compiled with a low wait limit and with CTA 0's
// value tile `g_withheld` never handed over.  Nothing is in flight for what is
// withheld.
#include <string.h>

#include "common.cuh"
__device__ int g_withheld = -1;
#include "kv_prefill.cuh"

using namespace nvfp4;

template <int MODE>
static cudaError_t launch(const kv::AttnArgs& a, unsigned grid, cudaStream_t stream) {
  auto kern = kv::pf::k_kv_prefill<__nv_bfloat16, MODE, 64, true>;
  constexpr int smem = (int)kv::pf::Shape<MODE, 64>::smem;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, kv::pf::THREADS, smem, stream>>>(a);
  return cudaGetLastError();
}

extern "C" {

// B sequences of n drafts over L tokens of an NVFP4 (mode 0) or MXFP8 (1)
// cache without global scales, D = 64, a page a sequence, nothing split.
__attribute__((visibility("default"))) int kv_give_up(int mode, int withheld, void* k_codes, void* k_scales, void* v_codes, void* v_scales,
                                                      const void* q, const int32_t* q_start, const int32_t* kv_len, const int32_t* page_table,
                                                      const uint32_t* tree, void* out, float* lse, uint32_t B, uint32_t n, uint32_t L,
                                                      uint32_t heads, uint32_t G, uint32_t words, cudaStream_t stream) {
  const uint32_t D = 64;
  kv::AttnArgs a;
  memset(&a, 0, sizeof(a));
  a.codes[0] = static_cast<const uint8_t*>(k_codes);
  a.codes[1] = static_cast<const uint8_t*>(v_codes);
  a.scales[0] = static_cast<const uint8_t*>(k_scales);
  a.scales[1] = static_cast<const uint8_t*>(v_scales);
  a.q = q;
  a.q_stride = (int64_t)heads * G * D;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.page_table = page_table;
  a.out = out;
  a.lse = lse;
  a.scale = 0.125f;
  a.B = B;
  a.T = B * n;
  a.Hq = heads * G;
  a.heads = heads;
  a.G = G;
  a.D = D;
  a.max_q = n;
  a.max_kv = L;
  a.max_pages = 1;
  a.num_pages = B;
  a.page_size = L;
  a.tree = tree;
  a.tree_words = words;
  a.chunk = (int32_t)((L + 127) / 128 * 128);
  a.chunks = 1;
  a.tile_rows = 256;
  a.scale_bytes = (uint64_t)B * heads * L * (D / (mode == 0 ? 16 : 32));
  a.by_page.init(L);
  const unsigned grid = (n * G + 255u) / 256u * B * heads;
  cudaError_t e = cudaMemcpyToSymbol(g_withheld, &withheld, sizeof(withheld));
  if (e != cudaSuccess) return (int)e;
  e = mode == 0 ? launch<kv::kNV>(a, grid, stream) : launch<kv::kMX8>(a, grid, stream);
  return (int)e;
}

// Waits for the device; the error word (cleared), or minus a CUDA error.
__attribute__((visibility("default"))) int kv_give_up_word() {
  cudaError_t e = cudaDeviceSynchronize();
  unsigned word = 0, zero = 0;
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(&word, g_device_error, sizeof(word));
  if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero));
  return e == cudaSuccess ? (int)word : -(int)e;
}

}  // extern "C"
