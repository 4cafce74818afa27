// Pages of a paged INT4 KV cache copied to other pages (QuaRot reviews, final
// comments: the KV cache at 4 bits; the pages have no counterpart to moving
// its pages): for every (source, destination) pair, every layer and every
// array, page[destination] = page[source].
//
// Bound by HBM: each byte is read once and written once.  One CTA takes one
// (pair, layer) and a slice of the page; a thread keeps kUnroll 16-byte loads
// in flight before it stores.  The scale and zero-point pages are short (two
// bytes a token and head), so the first slice takes them along, in the widest
// unit that divides both a page's and a layer's bytes.
#include <cstdint>

#include "kq_internal.h"

namespace kq {
namespace kvc {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;

struct Params {
  const int32_t* pairs;
  uint8_t* codes[2];          // K and V, or K alone (arrays = 1)
  uint16_t* small_[4];        // K scales, K zeros, V scales, V zeros
  int arrays;
  int64_t pages;              // pages a layer
  int64_t n_pairs;
  int64_t code_page;          // bytes
  int64_t code_layer;
  int64_t small_page;
  int64_t small_layer;
  int small_unit;             // 2, 4, 8 or 16 bytes
};

template <class T>
__device__ __forceinline__ void copy_small(const Params& P, int64_t src, int64_t dst) {
  const int64_t units = P.small_page / (int64_t)sizeof(T);
  for (int64_t i = threadIdx.x; i < units * 2 * P.arrays; i += kThreads) {
    const int a = (int)(i / units);
    const int64_t o = (i - a * units) * (int64_t)sizeof(T);
    char* base = reinterpret_cast<char*>(P.small_[a]);
    *reinterpret_cast<T*>(base + dst + o) = *reinterpret_cast<const T*>(base + src + o);
  }
}

__global__ void __launch_bounds__(kThreads) k_copy_pages(Params P) {
  const int64_t layer = blockIdx.x / P.n_pairs, pair = blockIdx.x - layer * P.n_pairs;
  const int64_t s = P.pairs[2 * pair], d = P.pairs[2 * pair + 1];
  if (s < 0 || d < 0 || s >= P.pages || d >= P.pages || s == d) return;
  const int64_t units = P.code_page / 16;
  const int64_t src = layer * P.code_layer + s * P.code_page;
  const int64_t dst = layer * P.code_layer + d * P.code_page;
  for (int a = 0; a < P.arrays; ++a) {
    const uint4* from = reinterpret_cast<const uint4*>(P.codes[a] + src);
    uint4* to = reinterpret_cast<uint4*>(P.codes[a] + dst);
    for (int64_t u = (int64_t)blockIdx.y * (kThreads * kUnroll) + threadIdx.x; u < units;
         u += (int64_t)gridDim.y * (kThreads * kUnroll)) {
      uint4 v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (u + j * kThreads < units) v[j] = from[u + j * kThreads];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j)
        if (u + j * kThreads < units) to[u + j * kThreads] = v[j];
    }
  }
  if (blockIdx.y == 0) {
    const int64_t ss = layer * P.small_layer + s * P.small_page;
    const int64_t sd = layer * P.small_layer + d * P.small_page;
    switch (P.small_unit) {
      case 16: copy_small<uint4>(P, ss, sd); break;
      case 8: copy_small<uint2>(P, ss, sd); break;
      case 4: copy_small<uint32_t>(P, ss, sd); break;
      default: copy_small<uint16_t>(P, ss, sd); break;
    }
  }
}

}  // namespace kvc

cudaError_t launch_kv_copy(const int32_t* pairs, int64_t n_pairs, int page_size,
                           int64_t num_slots, int layers, int dim, uint8_t* const codes[2],
                           uint16_t* const small_[4], int arrays, cudaStream_t s) {
  kvc::Params P{};
  P.pairs = pairs;
  for (int a = 0; a < 2; ++a) P.codes[a] = codes[a];
  for (int a = 0; a < 4; ++a) P.small_[a] = small_[a];
  P.arrays = arrays;
  P.pages = num_slots / page_size;
  P.n_pairs = n_pairs;
  P.code_page = (int64_t)page_size * (dim / 2);
  P.code_layer = num_slots * (dim / 2);
  P.small_page = (int64_t)page_size * (dim / 128) * 2;
  P.small_layer = num_slots * (dim / 128) * 2;
  P.small_unit = 16;
  while (P.small_page % P.small_unit || P.small_layer % P.small_unit) P.small_unit /= 2;
  const int64_t slice = 16 * kvc::kThreads * kvc::kUnroll;
  int64_t slices = (P.code_page + slice - 1) / slice;
  if (slices > 1024) slices = 1024;
  kvc::k_copy_pages<<<dim3((unsigned)(n_pairs * layers), (unsigned)slices), kvc::kThreads, 0,
                      s>>>(P);
  return cudaGetLastError();
}

}  // namespace kq
