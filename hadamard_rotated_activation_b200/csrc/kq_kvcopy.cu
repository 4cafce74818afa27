// Pages of a paged INT4 KV cache copied to other pages (QuaRot reviews, final
// comments: the KV cache at 4 bits; the pages have no counterpart to moving
// its pages): for every (source, destination) pair, every layer and every
// array, page[destination] = page[source].
//
// Bound by HBM: each byte is read once and written once.  One CTA takes one
// (pair, layer) and a slice of the page.  All of a slice's loads -- kUnroll 16-byte
// pieces a thread of the key and of the value codes, and in the first slice the
// short scale and zero-point pages (two bytes a token and head, in the widest unit
// that divides both a page's and a layer's bytes) -- are on their way before the
// first store: 1500 pages of 16 tokens and 8 heads in 4 layers take 34.4 us (6.1
// TB/s, 0.93 of the copy rate; 35.4 with loads marked as read once), and took 56.6 with
// one array after the other.
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
__device__ __forceinline__ void copy_slice(const Params& P, int64_t src, int64_t dst, int64_t ssrc,
                                           int64_t sdst) {
  const int64_t units = P.code_page / 16, step = (int64_t)gridDim.y * (kThreads * kUnroll);
  int64_t u = (int64_t)blockIdx.y * (kThreads * kUnroll) + threadIdx.x;
  // the short arrays as one row of units, array after array
  const int64_t each = P.small_page / (int64_t)sizeof(T);
  const int64_t all = blockIdx.y == 0 ? each * 2 * P.arrays : 0;
  int64_t i = threadIdx.x;
  auto small_at = [&](int64_t base, int64_t at) {
    const bool vals = at >= 2 * each;
    at -= vals ? 2 * each : 0;
    const bool zero = at >= each;
    at -= zero ? each : 0;
    uint16_t* const sp = vals ? P.small_[2] : P.small_[0];
    uint16_t* const zp = vals ? P.small_[3] : P.small_[1];
    return reinterpret_cast<T*>(reinterpret_cast<char*>(zero ? zp : sp) + base) + at;
  };
  do {
    uint4 k[kUnroll], v[kUnroll];
    T t;
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (u + j * kThreads < units) {
        k[j] = __ldcg(reinterpret_cast<const uint4*>(P.codes[0] + src) + u + j * kThreads);
        if (P.arrays > 1)
          v[j] = __ldcg(reinterpret_cast<const uint4*>(P.codes[1] + src) + u + j * kThreads);
      }
    if (i < all) t = *small_at(ssrc, i);
#pragma unroll
    for (int j = 0; j < kUnroll; ++j)
      if (u + j * kThreads < units) {
        reinterpret_cast<uint4*>(P.codes[0] + dst)[u + j * kThreads] = k[j];
        if (P.arrays > 1) reinterpret_cast<uint4*>(P.codes[1] + dst)[u + j * kThreads] = v[j];
      }
    if (i < all) *small_at(sdst, i) = t;
    u += step;
    i += kThreads;
  } while (u - threadIdx.x < units || i - threadIdx.x < all);
}

__global__ void __launch_bounds__(kThreads) k_copy_pages(Params P) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const uint32_t layer = blockIdx.x / (uint32_t)P.n_pairs;
  const uint32_t pair = blockIdx.x - layer * (uint32_t)P.n_pairs;
  // in order with the wait; the pages' loads follow from it
  int2 sd;
  asm volatile("ld.global.v2.s32 {%0, %1}, [%2];"
               : "=r"(sd.x), "=r"(sd.y)
               : "l"(P.pairs + 2 * (int64_t)pair)
               : "memory");
  const int64_t s = sd.x, d = sd.y;
  if (s < 0 || d < 0 || s >= P.pages || d >= P.pages || s == d) return;
  const int64_t src = layer * P.code_layer + s * P.code_page;
  const int64_t dst = layer * P.code_layer + d * P.code_page;
  const int64_t ss = layer * P.small_layer + s * P.small_page;
  const int64_t ds = layer * P.small_layer + d * P.small_page;
  switch (P.small_unit) {
    case 16: copy_slice<uint4>(P, src, dst, ss, ds); break;
    case 8: copy_slice<uint2>(P, src, dst, ss, ds); break;
    case 4: copy_slice<uint32_t>(P, src, dst, ss, ds); break;
    default: copy_slice<uint16_t>(P, src, dst, ss, ds); break;
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
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg = dependent_launch(
      dim3((unsigned)(n_pairs * layers), (unsigned)slices), kvc::kThreads, 0, s, attr);
  return cudaLaunchKernelEx(&cfg, kvc::k_copy_pages, P);
}

}  // namespace kq
