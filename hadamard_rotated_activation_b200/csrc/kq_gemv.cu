// Products of a few tokens with a 4-bit weight matrix: the linear layer of a
// decode step (QuaRot reviews, review 3 Questions: X W^T is unchanged when both
// carry the rotation; NVFP4 thread, discrete_descent's note: INT4-g128, NVFP4
// and MXFP4 weights).
//   y[j][i] = sum_k x[j][k] w[i][k]
// One warp per weight row, 32 codes a lane and step, fp32 throughout.
#include <cstdint>
#include <cuda_bf16.h>

#include "kq.h"
#include "kq_internal.h"

namespace kq {
namespace gv {

constexpr int kWarps = 8;
constexpr int kMaxM = KQ_GEMV_MAX_TOKENS;

struct Params {
  const void* x;
  const uint8_t* codes;
  const void* scales;
  const void* zeros;
  const float* tscale;
  void* y;
  int64_t n;
  int m, k, fmt, x_bf16, y_bf16;
};

__global__ void __launch_bounds__(32 * kWarps) k_gemv(Params P) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= P.n) return;
  float acc[kMaxM] = {};
  for (int c = lane * 32; c < P.k; c += 32 * 32) {
    const uint4 q = *reinterpret_cast<const uint4*>(P.codes + row * (P.k / 2) + c / 2);
    const uint32_t w4[4] = {q.x, q.y, q.z, q.w};
    for (int e = 0; e < 32; ++e) {
      const uint32_t code = (w4[e >> 3] >> (4 * (e & 7))) & 15u;
      const int col = c + e;
      float w;
      if (P.fmt == KQ_FMT_INT4_SYM) {
        w = (float)((int)(code ^ 8u) - 8) * static_cast<const float*>(P.scales)[row];
      } else if (P.fmt == KQ_FMT_INT4_ASYM) {
        const int64_t g = row * (P.k / 128) + col / 128;
        w = ((float)code - f16_bits_to_f32(static_cast<const uint16_t*>(P.zeros)[g])) *
            f16_bits_to_f32(static_cast<const uint16_t*>(P.scales)[g]);
      } else if (P.fmt == KQ_FMT_NVFP4) {
        w = e2m1_decode(code) *
            e4m3_decode(static_cast<const uint8_t*>(P.scales)[row * (P.k / 16) + col / 16]);
      } else {
        w = ldexpf(e2m1_decode(code),
                   (int)static_cast<const uint8_t*>(P.scales)[row * (P.k / 32) + col / 32] - 127);
      }
      for (int j = 0; j < kMaxM; ++j)
        if (j < P.m) {
          const int64_t at = (int64_t)j * P.k + col;
          const float xv = P.x_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(P.x)[at])
                                    : static_cast<const float*>(P.x)[at];
          acc[j] = fmaf(xv, w, acc[j]);
        }
    }
  }
  const float t = P.fmt == KQ_FMT_NVFP4 ? *P.tscale : 1.0f;
  for (int j = 0; j < kMaxM; ++j) {
    if (j >= P.m) break;
    float v = acc[j];
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    v *= t;
    if (lane == 0) {
      const int64_t at = (int64_t)j * P.n + row;
      if (P.y_bf16)
        static_cast<__nv_bfloat16*>(P.y)[at] = __float2bfloat16_rn(v);
      else
        static_cast<float*>(P.y)[at] = v;
    }
  }
}

}  // namespace gv

cudaError_t launch_gemv(int fmt, const void* x, int x_bf16, int m, const uint8_t* codes,
                        const void* scales, const void* zeros, const float* tscale, int64_t n,
                        int k, void* y, int y_bf16, cudaStream_t s) {
  gv::Params P{x, codes, scales, zeros, tscale, y, n, m, k, fmt, x_bf16, y_bf16};
  gv::k_gemv<<<(unsigned)((n + gv::kWarps - 1) / gv::kWarps), 32 * gv::kWarps, 0, s>>>(P);
  return cudaGetLastError();
}

}  // namespace kq
