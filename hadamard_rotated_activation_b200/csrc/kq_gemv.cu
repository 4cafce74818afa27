// Products of a few tokens with a 4-bit weight matrix: the linear layer of a
// decode step (QuaRot reviews, review 3 Questions: X W^T is unchanged when both
// carry the rotation; NVFP4 thread, discrete_descent's note: INT4-g128, NVFP4
// and MXFP4 weights).
//   y[j][i] = sum_k x[j][k] w[i][k]
//
// Mathematics.  The contraction runs on the bare codes, with the tokens as
// columns of mma.sync (m16n8k16, fp16 operands, fp32 sums) and 16 weight rows
// as its rows:
//   INT4   a code masked out of its word is an fp16 number (u 2^-24, or
//          16 u 2^-24 for the upper nibble of a byte), so a word of 8 codes
//          costs 5 integer operations; the 16 is taken out of x.  Per group of
//          128: s (2^24 sum u x - z sum x); symmetric codes are u - 8.
//   NVFP4  E2M1 codes by the hardware conversion, times the block's E4M3 scale:
//          at most 6 significant bits, exact in fp16.
//   MXFP4  likewise, the block's power of two taken relative to the largest of
//          the row's four blocks in the group (exact down to 2^-23 of it).
// x is held per token and group of 128 as fp16 with a power of two that puts its
// largest element in [2^14, 2^15): bf16 rows are exact down to 2^-28 of it.
// fp32 rows are two columns, the rounded value and 2^11 times what it leaves.
// A group's sum leaves the tensor core after 8 steps and is added in fp32.
//
// Bound by HBM: every code is read once, m n k multiplications ride along.  One
// CTA takes R rows (16 a warp) and a range of k; the CTAs of a cluster share the
// rows, split k between them and join their sums through distributed shared
// memory in rank order, so there is no workspace, one launch and a fixed order
// of additions.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "kq.h"
#include "kq_internal.h"
#include "kq_sm100.cuh"

namespace kq {
namespace gv {

namespace cg = cooperative_groups;
using sm100::pow2f;
using sm100::redux_max;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBatch = 4;                 // groups a warp has in flight

struct Params {
  const void* x;
  const uint8_t* codes;
  const void* scales;
  const uint16_t* zeros;
  const float* tscale;
  void* y;
  int64_t n;
  int m, k, groups;                       // groups of 128 columns, the last may be short
  int x_bf16, y_bf16;
  int wr;                                 // warps along the rows; kWarps / wr along k
};

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
               "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Eight E2M1 codes -> four fp16 pairs, in the order of the codes.
__device__ __forceinline__ void e2m1_halves(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}
__device__ __forceinline__ uint32_t mul_h2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t half_bits(float v) {
  return __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float half_value(uint32_t h) {
  return __half2float(__ushort_as_half((unsigned short)h));
}

// Stages x of groups [g0, g0 + ng) for the columns of NT mma tiles.  A warp takes
// one (group, token), a lane 4 consecutive elements.  Fragment order: 16 bytes
// for every (group, tile, word j, column, t) hold the 8 elements 32 t + 8 j ...,
// as pairs (0,4) (1,5) (2,6) (3,7) for the masked INT4 codes, whose odd ones
// carry a factor 16, or in their own order for the converted E2M1 codes.
template <bool INT4, int NT>
__device__ __forceinline__ void stage_x(const Params& P, int g0, int ng, uint16_t* xs, float2* xf) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int i = warp; i < ng * P.m; i += kWarps) {
    const int gi = i / P.m, tok = i - gi * P.m;
    const int k0 = (g0 + gi) * 128 + 4 * lane;
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (k0 < P.k) {
      const int64_t at = (int64_t)tok * P.k + k0;
      if (P.x_bf16) {
        const uint2 w = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(P.x) + at));
        v[0] = __uint_as_float(w.x << 16);
        v[1] = __uint_as_float(w.x & 0xffff0000u);
        v[2] = __uint_as_float(w.y << 16);
        v[3] = __uint_as_float(w.y & 0xffff0000u);
      } else {
        const float4 w = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(P.x) + at));
        v[0] = w.x;
        v[1] = w.y;
        v[2] = w.z;
        v[3] = w.w;
      }
    }
    float top = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
    const uint32_t bits = redux_max(__float_as_uint(top));
    const int sh = bits ? min(14 - ((int)(bits >> 23) - 127), 126) : 0;
    const float up = pow2f(sh);
    for (int part = 0; part < (P.x_bf16 ? 1 : 2); ++part) {
      const int col = P.x_bf16 ? tok : 2 * tok + part;
      uint16_t h[4];
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (part == 0) v[e] *= up;
        h[e] = (uint16_t)half_bits(v[e]);
        const float r = half_value(h[e]);
        v[e] = (v[e] - r) * 2048.0f;
        sum += r;
        if (INT4 && (e & 1)) h[e] = (uint16_t)half_bits(r * 0.0625f);
      }
      const int t = lane >> 3, j = (lane >> 1) & 3;
      uint16_t* to = xs + (size_t)(((gi * NT + (col >> 3)) * 4 + j) * 32 + (col & 7) * 4 + t) * 8;
      if (INT4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) to[2 * e + (lane & 1)] = h[e];
      } else {
        *reinterpret_cast<uint2*>(to + 4 * (lane & 1)) =
            make_uint2(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16);
      }
      if (INT4) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      if (lane == 0)
        xf[gi * NT * 8 + col] = make_float2(part == 0 ? pow2f(-sh) : pow2f(-sh) * 0x1p-11f, sum);
    }
  }
}


template <int FMT, int NT>
__global__ void __launch_bounds__(kThreads) k_gemv(Params P) {
  constexpr bool INT4 = FMT == KQ_FMT_INT4_SYM || FMT == KQ_FMT_INT4_ASYM;
  extern __shared__ __align__(16) uint8_t smem[];
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = (int)cluster.block_rank(), ranks = (int)cluster.num_blocks();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int wk = kWarps / P.wr, wr_i = warp % P.wr, wk_i = warp / P.wr;
  const int chunk = kBatch * wk;          // groups staged at a time
  uint16_t* xs = reinterpret_cast<uint16_t*>(smem);
  float2* xf = reinterpret_cast<float2*>(smem + (size_t)chunk * NT * 2048);
  float* red = reinterpret_cast<float*>(xf + chunk * NT * 8);

  const int rows = 16 * P.wr;
  const int64_t row0 = (int64_t)(blockIdx.x / ranks) * rows;
  const int cols = P.x_bf16 ? P.m : 2 * P.m;
  const int64_t last = P.n - 1;
  const int64_t ra = min(row0 + 16 * wr_i + g, last), rb = min(row0 + 16 * wr_i + 8 + g, last);
  const uint8_t* ca = P.codes + ra * (P.k / 2) + 16 * t;
  const uint8_t* cb = P.codes + rb * (P.k / 2) + 16 * t;

  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;

  const int gend = (int)((int64_t)(rank + 1) * P.groups / ranks);
  for (int g0 = (int)((int64_t)rank * P.groups / ranks); g0 < gend; g0 += chunk) {
    const int ng = min(chunk, gend - g0);
    // ---- this warp's codes and scales: groups g0 + wk_i, + wk, ...
    uint4 wa[kBatch], wb[kBatch];
    uint32_t sa[kBatch], sb[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int gi = g0 + wk_i + i * wk;
      wa[i] = wb[i] = make_uint4(0, 0, 0, 0);
      sa[i] = sb[i] = 0;
      if (gi < gend && gi * 128 + 32 * t < P.k) {
        wa[i] = __ldg(reinterpret_cast<const uint4*>(ca + (int64_t)gi * 64));
        wb[i] = __ldg(reinterpret_cast<const uint4*>(cb + (int64_t)gi * 64));
        if (FMT == KQ_FMT_INT4_ASYM) {
          const uint16_t* s16 = static_cast<const uint16_t*>(P.scales);
          sa[i] = __ldg(s16 + ra * P.groups + gi) | (uint32_t)__ldg(P.zeros + ra * P.groups + gi) << 16;
          sb[i] = __ldg(s16 + rb * P.groups + gi) | (uint32_t)__ldg(P.zeros + rb * P.groups + gi) << 16;
        } else if (FMT == KQ_FMT_NVFP4) {
          const uint16_t* s16 = static_cast<const uint16_t*>(P.scales);
          sa[i] = __ldg(s16 + ra * (P.k / 32) + gi * 4 + t);
          sb[i] = __ldg(s16 + rb * (P.k / 32) + gi * 4 + t);
        } else if (FMT == KQ_FMT_MXFP4) {
          const uint8_t* s8 = static_cast<const uint8_t*>(P.scales);
          sa[i] = __ldg(s8 + ra * (P.k / 32) + gi * 4 + t);
          sb[i] = __ldg(s8 + rb * (P.k / 32) + gi * 4 + t);
        }
      }
    }
    __syncthreads();                      // the last chunk's x is no longer read
    stage_x<INT4, NT>(P, g0, ng, xs, xf);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int gl = wk_i + i * wk;       // group within the chunk
      if (gl >= ng) break;
      float c[NT][4];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int j = 0; j < 4; ++j) c[n][j] = 0.0f;
      const uint32_t xa[4] = {wa[i].x, wa[i].y, wa[i].z, wa[i].w};
      const uint32_t xb[4] = {wb[i].x, wb[i].y, wb[i].z, wb[i].w};
      uint32_t ea = 0, eb = 0;            // MXFP4: largest exponent byte of the row's blocks
      uint32_t ma[2] = {0, 0}, mb[2] = {0, 0};
      if (FMT == KQ_FMT_NVFP4) {
        // both blocks' E4M3 scales as fp16, each in both halves
        uint32_t ha, hb;
        asm("{.reg .b16 v; cvt.u16.u32 v, %1; cvt.rn.f16x2.e4m3x2 %0, v;}" : "=r"(ha) : "r"(sa[i]));
        asm("{.reg .b16 v; cvt.u16.u32 v, %1; cvt.rn.f16x2.e4m3x2 %0, v;}" : "=r"(hb) : "r"(sb[i]));
        ma[0] = __byte_perm(ha, 0, 0x1010);
        ma[1] = __byte_perm(ha, 0, 0x3232);
        mb[0] = __byte_perm(hb, 0, 0x1010);
        mb[1] = __byte_perm(hb, 0, 0x3232);
      } else if (FMT == KQ_FMT_MXFP4) {
        ea = max(sa[i], __shfl_xor_sync(0xffffffffu, sa[i], 1));
        ea = max(ea, __shfl_xor_sync(0xffffffffu, ea, 2));
        eb = max(sb[i], __shfl_xor_sync(0xffffffffu, sb[i], 1));
        eb = max(eb, __shfl_xor_sync(0xffffffffu, eb, 2));
        auto down = [](uint32_t d) {      // 2^-d in both halves
          const uint32_t h = d < 15 ? (15 - d) << 10 : d < 25 ? 1u << (24 - d) : 0u;
          return h | h << 16;
        };
        ma[0] = ma[1] = down(ea - sa[i]);
        mb[0] = mb[1] = down(eb - sb[i]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t fa[4], fb[4];
        if (INT4) {
          const uint32_t flip = FMT == KQ_FMT_INT4_SYM ? 0x88888888u : 0u;
          const uint32_t va = xa[j] ^ flip, vb = xb[j] ^ flip;
          fa[0] = va & 0x000f000fu;
          fa[1] = va & 0x00f000f0u;
          fa[2] = va >> 8 & 0x000f000fu;
          fa[3] = va >> 8 & 0x00f000f0u;
          fb[0] = vb & 0x000f000fu;
          fb[1] = vb & 0x00f000f0u;
          fb[2] = vb >> 8 & 0x000f000fu;
          fb[3] = vb >> 8 & 0x00f000f0u;
        } else {
          e2m1_halves(xa[j], fa);
          e2m1_halves(xb[j], fb);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            fa[e] = mul_h2(fa[e], ma[j >> 1]);
            fb[e] = mul_h2(fb[e], mb[j >> 1]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint4 b = make_uint4(0, 0, 0, 0);
          if (8 * n + g < cols)
            b = *reinterpret_cast<const uint4*>(xs + (size_t)(((gl * NT + n) * 4 + j) * 32 + lane) * 8);
          mma16816(c[n], fa[0], fb[0], fa[1], fb[1], b.x, b.y);
          mma16816(c[n], fa[2], fb[2], fa[3], fb[3], b.z, b.w);
        }
      }
      // ---- the group's sums, scaled and added in fp32
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float2 f[2];
        f[0] = xf[gl * NT * 8 + 8 * n + 2 * t];
        f[1] = xf[gl * NT * 8 + 8 * n + 2 * t + 1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 q = f[e & 1];
          if (8 * n + 2 * t + (e & 1) >= cols) continue;
          const uint32_t s = e < 2 ? sa[i] : sb[i];
          if (FMT == KQ_FMT_INT4_ASYM)
            acc[n][e] = fmaf(half_value(s & 0xffffu) * q.x,
                             fmaf(-half_value(s >> 16), q.y, c[n][e] * 0x1p24f), acc[n][e]);
          else if (FMT == KQ_FMT_INT4_SYM)
            acc[n][e] = fmaf(q.x, fmaf(-8.0f, q.y, c[n][e] * 0x1p24f), acc[n][e]);
          else if (FMT == KQ_FMT_NVFP4)
            acc[n][e] = fmaf(q.x, c[n][e], acc[n][e]);
          else {
            const uint32_t eb8 = e < 2 ? ea : eb;
            const float p = __uint_as_float(eb8 ? eb8 << 23 : 0x00400000u);
            acc[n][e] = fmaf(c[n][e] * q.x, p, acc[n][e]);
          }
        }
      }
    }
  }

  // ---- join: the warps along k and the cluster's CTAs, in order
  const int mt = P.m;
  {
    float* to = red + (size_t)(wk_i * rows + 16 * wr_i) * mt;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if (P.x_bf16) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int tok = 8 * n + 2 * t + (e & 1);
          if (tok < mt) to[(g + 8 * (e >> 1)) * mt + tok] = acc[n][e];
        }
      } else {
        const int tok = 4 * n + t;
        if (tok < mt) {
          to[g * mt + tok] = acc[n][0] + acc[n][1];
          to[(g + 8) * mt + tok] = acc[n][2] + acc[n][3];
        }
      }
    }
  }
  cluster.sync();
  for (int i = rank * kThreads + threadIdx.x; i < rows * mt; i += ranks * kThreads) {
    // consecutive threads: consecutive rows of one token
    const int tok = i / rows, r = i - tok * rows;
    const int64_t row = row0 + r;
    if (row >= P.n) continue;
    float v = 0.0f;
    for (int c = 0; c < ranks; ++c) {
      const float* from = cluster.map_shared_rank(red, c);
      for (int w = 0; w < wk; ++w) v += from[(size_t)(w * rows + r) * mt + tok];
    }
    if (FMT == KQ_FMT_INT4_SYM) v *= static_cast<const float*>(P.scales)[row];
    if (FMT == KQ_FMT_NVFP4) v *= *P.tscale;
    const int64_t at = (int64_t)tok * P.n + row;
    if (P.y_bf16)
      static_cast<__nv_bfloat16*>(P.y)[at] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(P.y)[at] = v;
  }
  cluster.sync();                         // the others may still read this CTA's sums
}

template <int FMT, int NT>
cudaError_t launch(Params P, cudaStream_t s) {
  int ranks = 1;
  P.wr = 8;
  const int64_t blocks = (P.n + 16 * P.wr - 1) / (16 * P.wr);
  while (ranks < 8 && blocks * ranks < 3 * 148 && P.groups / (2 * ranks) >= kBatch) ranks *= 2;
  const int wk = kWarps / P.wr, chunk = kBatch * wk;
  const size_t smem = (size_t)chunk * NT * (2048 + 64) + sizeof(float) * wk * 16 * P.wr * P.m;
  cudaError_t e = cudaFuncSetAttribute((const void*)k_gemv<FMT, NT>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks * ranks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_gemv<FMT, NT>, P);
}

template <int FMT>
cudaError_t launch_tiles(const Params& P, cudaStream_t s) {
  const int cols = P.x_bf16 ? P.m : 2 * P.m;
  if (cols <= 8) return launch<FMT, 1>(P, s);
  if (cols <= 16) return launch<FMT, 2>(P, s);
  return launch<FMT, 4>(P, s);
}

}  // namespace gv

cudaError_t launch_gemv(int fmt, const void* x, int x_bf16, int m, const uint8_t* codes,
                        const void* scales, const void* zeros, const float* tscale, int64_t n,
                        int k, void* y, int y_bf16, cudaStream_t s) {
  const gv::Params P{x, codes, scales, static_cast<const uint16_t*>(zeros), tscale, y, n, m, k,
                     (k + 127) / 128, x_bf16, y_bf16, 0};
  switch (fmt) {
    case KQ_FMT_INT4_SYM: return gv::launch_tiles<KQ_FMT_INT4_SYM>(P, s);
    case KQ_FMT_INT4_ASYM: return gv::launch_tiles<KQ_FMT_INT4_ASYM>(P, s);
    case KQ_FMT_NVFP4: return gv::launch_tiles<KQ_FMT_NVFP4>(P, s);
    default: return gv::launch_tiles<KQ_FMT_MXFP4>(P, s);
  }
}

}  // namespace kq
