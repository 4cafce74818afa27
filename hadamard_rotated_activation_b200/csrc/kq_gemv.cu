// Products of a few tokens with a 4-bit weight matrix: the linear layer of a
// decode step (QuaRot reviews, review 3 Questions: X W^T is unchanged when both
// carry the rotation; NVFP4 thread, discrete_descent's note: INT4-g128, NVFP4
// and MXFP4 weights).
//   y[j][i] = sum_k x[j][k] w[i][k]
//
// Mathematics.  The contraction runs on the bare codes, with the tokens as
// columns of mma.sync (m16n8k16, fp16 operands, fp32 sums) and 16 weight rows
// as its rows:
//   INT4, bf16 result: a code masked out of its word is an fp16 number (u 2^-24,
//          or 16 u 2^-24 for the upper nibble of a byte), so a word of 8 codes
//          costs 5 integer operations; the 16 is taken out of x.  Per group of
//          128: s (2^24 sum u x - z sum x); symmetric codes are u - 8.  The tensor
//          core lines up such subnormal operands as if they were 2^-14, which
//          costs 6 to 10 of its 25 bits: results are off by 5e-6, far inside bf16.
//   INT4, fp32 result: the masked code under the exponent of 1024, then 4 fp16
//          operations a word that take 1024 and the offset 8 away again: u - 8,
//          exactly, in full alignment (off by 2e-7); z - 8 takes the place of z.
//   NVFP4  E2M1 codes by the hardware conversion, times the block's E4M3 scale:
//          at most 6 significant bits, exact in fp16.
//   MXFP4  up to 8 columns: the block's sum leaves the tensor core and takes its power
//          of two in fp32.  More: as NVFP4, the power of two taken relative to the
//          largest of the row's four blocks in the group (exact down to 2^-23 of it).
// x is held per token and group of 128 as fp16 with a power of two that puts its
// largest element in [2^14, 2^15): bf16 rows are exact down to 2^-31 of it, and off by at
// most 2^-39 of it below (INT4 with a bf16 result, where every second pair is divided by
// 16: 2^-27 and 2^-35).  The largest sum, of E2M1 codes with their block scales, is below 2^34.
// fp32 rows are two columns, the rounded value and 2^11 times what it leaves.
// A group's sum leaves the tensor core after 8 steps and is added in fp32.
//
// Bound by HBM: every code is read once, m n k multiplications ride along.  The
// CTAs of a cluster share the rows, split k between them and join their sums through
// distributed shared memory in a fixed order, so there is no workspace and one
// launch.  Measured (one B200, time between calls in a graph), INT4 asymmetric:
// 4096 x 4096 by 1 token 5.0 us, 12288 x 4096 by 8 tokens 11.2 us; MXFP4 32003 x 4096
// by 4 tokens 21.3 us = 3.3 TB/s; NVFP4 4096 x 12288 by 2 fp32 tokens 9.9 us.  When the
// second took 11.9 us, about 2 were the launch, 1 the start, 2 staging x (which every
// CTA does for its range of k), 4 the products at 1.9 instructions a cycle, 1 the
// cluster barrier and 0.7 the join; with no copies at all it took 10.9.  When the third
// took 23.1, 15.5 remained without the products: there the memory and the instructions
// of the E2M1 conversion and the block scales share the bound.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>
#include <type_traits>

#include "kq.h"
#include "kq_internal.h"
#include "kq_mma16.cuh"
#include "kq_sm100.cuh"

namespace kq {
namespace gv {

namespace cg = cooperative_groups;
using namespace sm100;

// A warp streams its rows in steps of 16 rows by kStep groups, kStages of which are
// on their way or in use.  One tile of 8 columns: two CTAs of 8 warps an SM.  More:
// one CTA of 16 warps, which stages x once an SM, and shorter steps, which leave x
// and the sums more room (32000 x 4096 by 16 tokens takes 34 us and took 79 with two CTAs).
template <int NT>
struct Shape {
  static constexpr int kWarps = NT == 1 ? 8 : 16;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = NT == 1 ? 2 : 1;
  static constexpr int kStep = NT == 1 ? 4 : 2;
  static constexpr int kStages = NT == 1 ? 2 : 3;
  static constexpr int kRow = kStep * 64;             // bytes of a staged row of codes
  static constexpr int kScaleRow = kStep * 8;         // bytes of its scales at most
  static constexpr int kStage = 16 * (kRow + kScaleRow);
};

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
  int tiles, round;                       // 16-row tiles of a cluster, and of a round
  int seg;                                // groups whose x is staged at a time
  int parts, part_shift, part;            // warps that share a tile's groups: 2^part_shift, steps
                                          // of each
  int ranks, rank_shift;                  // CTAs of a cluster, which split k: 2^rank_shift
  int wide;                               // scales of a step's row by aligned copies
  uint32_t recip;                         // 2^16 / m, rounded up
};

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
__device__ __forceinline__ uint32_t add_h2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t fma_h2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ float half_value(uint32_t h) {
  return __half2float(__ushort_as_half((unsigned short)h));
}

template <int BYTES>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool in = true) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;"
                 :: "r"(dst), "l"(src), "n"(BYTES) : "memory");
}
// Eight INT4 codes (offset codes: symmetric ones with their sign bit turned) -> u - 8
// as fp16 pairs (0,4) (1,5) (2,6) (3,7).
template <bool TURN>
__device__ __forceinline__ void code_halves(uint32_t w, uint32_t (&h)[4]) {
  // Integers below 2^10 placed under the exponent of 1024 (the usual way from bits to a
  // floating-point number): 1024 + u and 1024 + 16 u, then - 1032 and / 16 - 72: every step is exact
  constexpr uint32_t lo = TURN ? 0x64086408u : 0x64006400u, hi = TURN ? 0x64806480u : 0x64006400u;
  const uint32_t v = w >> 8;
  h[0] = add_h2((w & 0x000f000fu) ^ lo, 0xe408e408u);
  h[1] = fma_h2((w & 0x00f000f0u) ^ hi, 0x2c002c00u, 0xd480d480u);
  h[2] = add_h2((v & 0x000f000fu) ^ lo, 0xe408e408u);
  h[3] = fma_h2((v & 0x00f000f0u) ^ hi, 0x2c002c00u, 0xd480d480u);
}

// Eight elements of a row of x as loaded.
struct Eight {
  uint4 a, b;
};
__device__ __forceinline__ Eight load8(const Params& P, int tok, int k0) {
  Eight e{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (tok < P.m && k0 < P.k) {
    const int64_t at = (int64_t)tok * P.k + k0;
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(P.x) +
                                                    at * (P.x_bf16 ? 2 : 4));
    e.a = p[0];
    if (!P.x_bf16) e.b = p[1];
  }
  return e;
}

// Stages x of groups [g0, g0 + ng) for the columns of NT mma tiles.  16 lanes take
// one (group, token), a lane 8 consecutive elements, which are one 16-byte piece
// in fragment order: (group, tile, word j, column, t) holds elements 32 t + 8 j ...
// as pairs (0,4) (1,5) (2,6) (3,7) for the masked INT4 codes (PAIRS), whose odd ones
// carry a factor 16 when they are taken as they are (SMALL), or in their own order
// for the converted E2M1 codes.  SUMS: the groups' sums too.  Columns
// behind the last one are left as they are: what they hold reaches no other
// column, and their sums are not stored.
template <int NT>
__device__ __forceinline__ Eight load_x(const Params& P, int g0, int ng, int round) {
  const int i = (threadIdx.x >> 4) + round * (Shape<NT>::kThreads / 16);
  const int gi = (int)(i * P.recip >> 16), tok = i - gi * P.m;
  return load8(P, i < ng * P.m ? tok : P.m, (g0 + gi) * 128 + 8 * (threadIdx.x & 15));
}
// `first`: what load_x gave for round 0, loaded before the codes' copies.
template <bool SMALL, bool SUMS, bool BLOCKS, bool PAIRS, int NT>
__device__ __forceinline__ void stage_x(const Params& P, int g0, int ng, const Eight& first,
                                        uint4* xs, float2* xf) {
  constexpr int kAhead = 4, kThreads = Shape<NT>::kThreads;
  const int lane16 = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int items = ng * P.m;
  const int rounds = (items + kThreads / 16 - 1) / (kThreads / 16);
#pragma unroll 1
  for (int r0 = 0; r0 < rounds; r0 += kAhead) {
    Eight in[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      in[u] = first;
      if (r0 + u > 0 && r0 + u < rounds) in[u] = load_x<NT>(P, g0, ng, r0 + u);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (r0 + u >= rounds) break;
      const int i = slot + (r0 + u) * (kThreads / 16);
      const int gi = (int)(i * P.recip >> 16), tok = i - gi * P.m;
      float v[8];
      if (P.x_bf16) {
        const uint32_t w[4] = {in[u].a.x, in[u].a.y, in[u].a.z, in[u].a.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[2 * e] = __uint_as_float(w[e] << 16);
          v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
        }
      } else {
        const uint32_t w[8] = {in[u].a.x, in[u].a.y, in[u].a.z, in[u].a.w,
                               in[u].b.x, in[u].b.y, in[u].b.z, in[u].b.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(w[e]);
      }
      float top = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[e]));
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // -113 to 126, -114 for an infinity
      const int sh = top > 0.0f ? min(141 - (int)(__float_as_uint(top) >> 23), 126) : 0;
      const float up = pow2f(sh);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] *= up;
        sum += v[e];
      }
      if (SUMS) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      if (i < items) {
        // block by block, a lane's 8 elements of block j begin at 32 j + 8 t
        const int t = BLOCKS ? lane16 & 3 : lane16 >> 2, j = BLOCKS ? lane16 >> 2 : lane16 & 3;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (part == 1 && P.x_bf16) break;
          const int col = P.x_bf16 ? tok : 2 * tok + part;
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& lo = v[PAIRS ? e : 2 * e];
            float& hi = v[PAIRS ? e + 4 : 2 * e + 1];
            h[e] = half2_bits(lo, hi);
            if (!P.x_bf16 && part == 0) {
              const float2 r = half2_floats(h[e]);
              lo = (lo - r.x) * 2048.0f;
              hi = (hi - r.y) * 2048.0f;
            }
            if (SMALL && (e & 1)) h[e] = mul_h2(h[e], 0x2c002c00u);   // / 16
          }
          xs[((gi * NT + (col >> 3)) * 4 + j) * 32 + (col & 7) * 4 + t] =
              make_uint4(h[0], h[1], h[2], h[3]);
          // the sum of the group (of both parts at once) rides on the first column
          if (lane16 == 0)
            xf[gi * NT * 8 + col] = part == 0 ? make_float2(pow2f(-sh), SMALL ? sum * 0x1p-24f : sum)
                                              : make_float2(pow2f(-sh) * 0x1p-11f, 0.0f);
        }
      }
    }
  }
}

// First group of a rank (ranks is a power of two): whole steps, so that the scales of a
// step's row are an aligned copy wherever the row's are.
template <int NT>
__device__ __forceinline__ int rank_begin(const Params& P, int rank) {
  constexpr int kStep = Shape<NT>::kStep;
  const uint32_t steps = (uint32_t)(P.groups + kStep - 1) / kStep;
  return min((int)(rank * steps >> P.rank_shift) * kStep, P.groups);
}

// Whether a format's blocks are summed one by one (MXFP4 with few columns): a
// block's two mma steps leave the tensor core and are scaled in fp32, which costs
// 16 multiply-adds a group and tile of 8 columns instead of 32 products of codes
// and scales.
template <int FMT, int NT>
constexpr bool kByBlock = FMT == KQ_FMT_MXFP4 && NT == 1;

// Where the 16-byte piece c of row r is staged.  Fragment reads take four pieces of
// two neighbouring rows at a time, or, block by block, 4 bytes of one piece of eight
// rows; either order has no bank conflicts.
template <bool BLOCKS>
__device__ __forceinline__ int piece(int r, int c) {
  return 16 * (c ^ (BLOCKS ? r & 7 : (r & 1) << 2));
}

// A warp's stream through the codes: the rows it is at, and the lane's share of
// the copies of a step (4 kStep lanes a row).
template <int FMT, int NT>
struct Stream {
  using S = Shape<NT>;
  static constexpr bool BLOCKS = kByBlock<FMT, NT>;
  static constexpr int LANES = 4 * S::kStep, ROWS = 32 / LANES;   // lanes a row, rows at a time
  const uint8_t* codes;                   // row0, the lane's piece
  const uint8_t* scales;                  // the lane's row of scales (zero points)
  int off[16 / ROWS];                     // bytes to the lane's rows (the last row again behind it)
  int64_t row0;

  __device__ __forceinline__ void start(const Params& P, int64_t row) {
    const int lane = threadIdx.x & 31;
    const int left = (int)min(P.n - 1 - row, (int64_t)15);
    row0 = row;
    codes = P.codes + row * (P.k / 2) + 16 * (lane % LANES);
#pragma unroll
    for (int i = 0; i < 16 / ROWS; ++i) off[i] = min(left, ROWS * i + lane / LANES) * (P.k / 2);
    const int64_t sr = row + min(left, lane & 15);
    if (FMT == KQ_FMT_INT4_ASYM)
      scales = reinterpret_cast<const uint8_t*>(
          (lane < 16 ? static_cast<const uint16_t*>(P.scales) : P.zeros) + sr * P.groups);
    else if (FMT == KQ_FMT_NVFP4)
      scales = static_cast<const uint8_t*>(P.scales) + sr * (P.k / 16) + 16 * (lane >> 4);
    else if (FMT == KQ_FMT_MXFP4)
      scales = static_cast<const uint8_t*>(P.scales) + sr * (P.k / 32);
  }

  // Starts the copies of groups g0 ... (none at or behind gend) into a stage: codes,
  // behind them 16 rows of scales: INT4 asymmetric kStep fp16 scales and zero
  // points, NVFP4 8 E4M3 bytes a group, MXFP4 4 E8M0 bytes a group.
  __device__ __forceinline__ void copy(const Params& P, int g0, int gend, uint8_t* stage) const {
    constexpr int kStep = S::kStep;
    const int lane = threadIdx.x & 31, c = lane % LANES, r = lane / LANES;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(stage);
    const bool in = g0 + (c >> 2) < gend && g0 * 128 + 32 * c < P.k;
    const uint8_t* from = codes + (in ? g0 * 64 : 0);
#pragma unroll
    for (int i = 0; i < 16 / ROWS; ++i)
      copy_async<16>(to + (ROWS * i + r) * S::kRow + piece<BLOCKS>(ROWS * i + r, c), from + off[i],
                     in);
    if (FMT == KQ_FMT_INT4_SYM) return;
    const uint32_t ts = to + 16 * S::kRow + (lane & 15) * S::kScaleRow;
    if (P.wide) {
      if (FMT == KQ_FMT_INT4_ASYM)
        copy_async<2 * kStep>(ts + (lane >> 4) * 2 * kStep, scales + 2 * g0);
      else if (FMT == KQ_FMT_NVFP4) {
        if (lane < 8 * kStep) copy_async<16>(ts + (lane >> 4) * 16, scales + 8 * g0);
      } else if (lane < 16) {
        copy_async<4 * kStep>(ts, scales + 4 * g0);
      }
      return;
    }
    // scales that no aligned copy reaches: one by one
    constexpr int per = FMT == KQ_FMT_INT4_ASYM ? 1 : FMT == KQ_FMT_NVFP4 ? 8 : 4;   // a group
    constexpr int kTurns = 16 * kStep * per / 32, kAhead = kTurns < 8 ? kTurns : 8;
    const int count = FMT == KQ_FMT_INT4_ASYM ? P.groups : FMT == KQ_FMT_NVFP4 ? P.k / 16 : P.k / 32;
    const int left = (int)min(P.n - 1 - row0, (int64_t)15);
#pragma unroll 1
    for (int j0 = 0; j0 < kTurns; j0 += kAhead) {
      uint16_t v[kAhead], z[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = lane + 32 * (j0 + j), row = i / (kStep * per), e = i - row * (kStep * per);
        const int at = g0 * per + e;
        const int64_t src = (row0 + min(left, row)) * count + at;
        const bool ok = at < gend * per && at < count;
        v[j] = z[j] = 0;
        if (FMT == KQ_FMT_INT4_ASYM) {
          if (ok) v[j] = static_cast<const uint16_t*>(P.scales)[src];
          if (ok) z[j] = P.zeros[src];
        } else if (ok) {
          v[j] = static_cast<const uint8_t*>(P.scales)[src];
        }
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int i = lane + 32 * (j0 + j), row = i / (kStep * per), e = i - row * (kStep * per);
        uint8_t* d = stage + 16 * S::kRow + row * S::kScaleRow;
        if (FMT == KQ_FMT_INT4_ASYM) {
          reinterpret_cast<uint16_t*>(d)[e] = v[j];
          reinterpret_cast<uint16_t*>(d)[kStep + e] = z[j];
        } else {
          d[e] = (uint8_t)v[j];
        }
      }
    }
  }
};

// 2^e for -127 <= e <= 128 as two factors.  With a group's sum c (0 or 2^-25 .. 2^27) and
// a token's scale f, c near f rest leaves fp32's range on the way only where the
// product does, whichever of the two scales is far from 1.
struct Power {
  float near, rest;
};
__device__ __forceinline__ Power power(int e) {
  const int h = max(min(e, 100), -100);
  return Power{pow2f(h), pow2f(e - h)};
}

// Adds a staged step: its first ng groups, times groups gl ... of the staged x.
template <int FMT, int NT, bool SMALL>
__device__ __forceinline__ void compute_step(const uint8_t* stage, int gl, int ng, const uint4* xs,
                                             const float2* xf, float (&acc)[NT][4]) {
  constexpr bool INT4 = FMT == KQ_FMT_INT4_SYM || FMT == KQ_FMT_INT4_ASYM;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  using S = Shape<NT>;
  constexpr int kStep = S::kStep, kRow = S::kRow, kScaleRow = S::kScaleRow;
  constexpr bool BLOCKS = kByBlock<FMT, NT>;
  const uint8_t* ca = stage + g * kRow;
  const uint8_t* sca = stage + 16 * kRow + g * kScaleRow;
  constexpr int kDown = 8 * kScaleRow;            // from row g to row g + 8
  const uint4* xg = xs + gl * NT * 128 + lane;
  const float2* fg = xf + gl * NT * 8 + 2 * t;
  // plain: sums of 2^(e - 127) c_b stay far inside fp32 (MXFP4 block by block)
  auto group = [&](int i, auto plain) {
    if constexpr (BLOCKS) {
      // block b: 8 codes a lane; 2^(e - 127) c_b of the four blocks, then the token's scale
      const uint32_t ea = *reinterpret_cast<const uint32_t*>(sca + 4 * i);
      const uint32_t eb = *reinterpret_cast<const uint32_t*>(sca + kDown + 4 * i);
      const float4 f = *reinterpret_cast<const float4*>(fg);
      auto block = [&](int b, float (&c)[4]) {
        const int at = piece<true>(g, 4 * i + b) + 4 * t;
        uint32_t fa[4], fb[4];
        e2m1_halves(*reinterpret_cast<const uint32_t*>(ca + at), fa);
        e2m1_halves(*reinterpret_cast<const uint32_t*>(ca + 8 * kRow + at), fb);
        const uint4 x = xg[b * 32];
        mma16816(c, fa[0], fb[0], fa[1], fb[1], x.x, x.y);
        mma16816(c, fa[2], fb[2], fa[3], fb[3], x.z, x.w);
      };
      if constexpr (plain) {
        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          block(b, c);
          const float pa = __uint_as_float(ea >> (8 * b) << 24 >> 1);
          const float pb = __uint_as_float(eb >> (8 * b) << 24 >> 1);
          sum[0] = fmaf(pa, c[0], sum[0]);
          sum[1] = fmaf(pa, c[1], sum[1]);
          sum[2] = fmaf(pb, c[2], sum[2]);
          sum[3] = fmaf(pb, c[3], sum[3]);
        }
        acc[0][0] = fmaf(f.x, sum[0], acc[0][0]);
        acc[0][1] = fmaf(f.z, sum[1], acc[0][1]);
        acc[0][2] = fmaf(f.x, sum[2], acc[0][2]);
        acc[0][3] = fmaf(f.z, sum[3], acc[0][3]);
      } else {
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          block(b, c);
          const Power pa = power((int)(ea >> (8 * b) & 255u) - 127);
          const Power pb = power((int)(eb >> (8 * b) & 255u) - 127);
          acc[0][0] = fmaf(c[0] * pa.near * f.x, pa.rest, acc[0][0]);
          acc[0][1] = fmaf(c[1] * pa.near * f.z, pa.rest, acc[0][1]);
          acc[0][2] = fmaf(c[2] * pb.near * f.x, pb.rest, acc[0][2]);
          acc[0][3] = fmaf(c[3] * pb.near * f.z, pb.rest, acc[0][3]);
        }
      }
      return;
    }
    const int at = piece<false>(g, 4 * i + t);
    const uint4 wa = *reinterpret_cast<const uint4*>(ca + at);
    const uint4 wb = *reinterpret_cast<const uint4*>(ca + 8 * kRow + at);
    const uint32_t xa[4] = {wa.x, wa.y, wa.z, wa.w}, xb[4] = {wb.x, wb.y, wb.z, wb.w};
    float c[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[n][j] = 0.0f;
    uint32_t ma[2] = {0, 0}, mb[2] = {0, 0};
    float sa = 1.0f, sb = 1.0f, za = 0.0f, zb = 0.0f;
    uint32_t ea = 0, eb = 0;                // MXFP4: the rows' largest block exponents
    if (FMT == KQ_FMT_INT4_ASYM) {
      const uint16_t* s16 = reinterpret_cast<const uint16_t*>(sca) + i;
      sa = half_value(s16[0]);
      za = half_value(s16[kStep]);
      sb = half_value(s16[kDown / 2]);
      zb = half_value(s16[kDown / 2 + kStep]);
      if (!SMALL) {
        za -= 8.0f;
        zb -= 8.0f;
      }
    } else if (FMT == KQ_FMT_INT4_SYM) {
      za = zb = SMALL ? 8.0f : 0.0f;
    } else if (FMT == KQ_FMT_NVFP4) {
      // both blocks' E4M3 scales as fp16, each in both halves
      const uint32_t ba = *reinterpret_cast<const uint16_t*>(sca + 8 * i + 2 * t);
      const uint32_t bb = *reinterpret_cast<const uint16_t*>(sca + kDown + 8 * i + 2 * t);
      uint32_t ha, hb;
      asm("{.reg .b16 v; cvt.u16.u32 v, %1; cvt.rn.f16x2.e4m3x2 %0, v;}" : "=r"(ha) : "r"(ba));
      asm("{.reg .b16 v; cvt.u16.u32 v, %1; cvt.rn.f16x2.e4m3x2 %0, v;}" : "=r"(hb) : "r"(bb));
      ma[0] = __byte_perm(ha, 0, 0x1010);
      ma[1] = __byte_perm(ha, 0, 0x3232);
      mb[0] = __byte_perm(hb, 0, 0x1010);
      mb[1] = __byte_perm(hb, 0, 0x3232);
    } else {
      // relative to the largest of the row's four blocks
      const uint32_t ba = sca[4 * i + t], bb = sca[kDown + 4 * i + t];
      ea = max(ba, __shfl_xor_sync(0xffffffffu, ba, 1));
      eb = max(bb, __shfl_xor_sync(0xffffffffu, bb, 1));
      ea = max(ea, __shfl_xor_sync(0xffffffffu, ea, 2));
      eb = max(eb, __shfl_xor_sync(0xffffffffu, eb, 2));
      auto down = [](uint32_t d) {        // 2^-d in both halves, 0 for d > 24
        const float f = __uint_as_float((127u - min(d, 100u)) << 23);
        return half2_bits(f, f);
      };
      ma[0] = ma[1] = down(ea - ba);
      mb[0] = mb[1] = down(eb - bb);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t fa[4], fb[4];
      if (INT4 && !SMALL) {
        code_halves<FMT == KQ_FMT_INT4_SYM>(xa[j], fa);
        code_halves<FMT == KQ_FMT_INT4_SYM>(xb[j], fb);
      } else if (INT4) {
        // symmetric codes are offset by 8
        constexpr uint32_t lo = FMT == KQ_FMT_INT4_SYM ? 0x00080008u : 0u, hi = lo << 4;
        fa[0] = (xa[j] & 0x000f000fu) ^ lo;
        fa[1] = (xa[j] & 0x00f000f0u) ^ hi;
        fa[2] = (xa[j] >> 8 & 0x000f000fu) ^ lo;
        fa[3] = (xa[j] >> 8 & 0x00f000f0u) ^ hi;
        fb[0] = (xb[j] & 0x000f000fu) ^ lo;
        fb[1] = (xb[j] & 0x00f000f0u) ^ hi;
        fb[2] = (xb[j] >> 8 & 0x000f000fu) ^ lo;
        fb[3] = (xb[j] >> 8 & 0x00f000f0u) ^ hi;
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
        const uint4 b = xg[(n * 4 + j) * 32];
        mma16816(c[n], fa[0], fb[0], fa[1], fb[1], b.x, b.y);
        mma16816(c[n], fa[2], fb[2], fa[3], fb[3], b.z, b.w);
      }
    }
    // ---- the group's sums, scaled and added in fp32
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4 f = *reinterpret_cast<const float4*>(fg + 8 * n);
      if (INT4) {
        acc[n][0] = fmaf(sa * f.x, fmaf(-za, f.y, c[n][0]), acc[n][0]);
        acc[n][1] = fmaf(sa * f.z, fmaf(-za, f.w, c[n][1]), acc[n][1]);
        acc[n][2] = fmaf(sb * f.x, fmaf(-zb, f.y, c[n][2]), acc[n][2]);
        acc[n][3] = fmaf(sb * f.z, fmaf(-zb, f.w, c[n][3]), acc[n][3]);
      } else if (FMT == KQ_FMT_NVFP4) {
        acc[n][0] = fmaf(f.x, c[n][0], acc[n][0]);
        acc[n][1] = fmaf(f.z, c[n][1], acc[n][1]);
        acc[n][2] = fmaf(f.x, c[n][2], acc[n][2]);
        acc[n][3] = fmaf(f.z, c[n][3], acc[n][3]);
      } else if (ea - 64u < 128u && eb - 64u < 128u) {
        // c 2^(e - 127) stays far inside fp32
        const float pa = __uint_as_float(ea << 23), pb = __uint_as_float(eb << 23);
        acc[n][0] = fmaf(f.x, c[n][0] * pa, acc[n][0]);
        acc[n][1] = fmaf(f.z, c[n][1] * pa, acc[n][1]);
        acc[n][2] = fmaf(f.x, c[n][2] * pb, acc[n][2]);
        acc[n][3] = fmaf(f.z, c[n][3] * pb, acc[n][3]);
      } else {
        const Power pa = power((int)ea - 127), pb = power((int)eb - 127);
        acc[n][0] = fmaf(c[n][0] * pa.near * f.x, pa.rest, acc[n][0]);
        acc[n][1] = fmaf(c[n][1] * pa.near * f.z, pa.rest, acc[n][1]);
        acc[n][2] = fmaf(c[n][2] * pb.near * f.x, pb.rest, acc[n][2]);
        acc[n][3] = fmaf(c[n][3] * pb.near * f.z, pb.rest, acc[n][3]);
      }
    }
  };
  // Exponents 64 .. 191 (the two top bits differ) in all four blocks of a row's group.
  auto plain_scales = [](uint32_t a) { return a ^ a << 1; };
  auto all_plain = [](uint32_t a) {
    return (bool)__all_sync(0xffffffffu, (a & 0x80808080u) == 0x80808080u);
  };
  // whole steps without a branch between groups
  bool whole = NT == 1 && ng >= kStep;
  if constexpr (BLOCKS) {
    static_assert(kStep == 4, "one load a row");
    const uint4 a = *reinterpret_cast<const uint4*>(sca);
    const uint4 b = *reinterpret_cast<const uint4*>(sca + kDown);
    const uint32_t in = plain_scales(a.x) & plain_scales(a.y) & plain_scales(a.z) &
                        plain_scales(a.w) & plain_scales(b.x) & plain_scales(b.y) &
                        plain_scales(b.z) & plain_scales(b.w);
    whole = all_plain(whole ? in : 0u);
  }
  if (whole) {
#pragma unroll
    for (int i = 0; i < kStep; ++i, xg += NT * 128, fg += NT * 8) group(i, std::true_type{});
  } else if (NT == 1) {
    const int n = min(ng, kStep);
#pragma unroll 1
    for (int i = 0; i < n; ++i, xg += NT * 128, fg += NT * 8) {
      if (BLOCKS && !all_plain(plain_scales(*reinterpret_cast<const uint32_t*>(sca + 4 * i)) &
                               plain_scales(*reinterpret_cast<const uint32_t*>(sca + kDown + 4 * i))))
        group(i, std::false_type{});
      else
        group(i, std::true_type{});
    }
  } else {
#pragma unroll
    for (int i = 0; i < kStep; ++i, xg += NT * 128, fg += NT * 8) {
      if (i >= ng) break;
      group(i, std::true_type{});
    }
  }
}

// A cluster takes 16 P.tiles rows and all of k, a CTA of it a range of k, a warp
// (tile, part) units: a tile by its part of the range.  Each warp keeps kStages
// steps of its units on their way by asynchronous copies into shared memory, with
// no barrier between warps; x of the range is staged once (in segments where k is
// long) while the first ones come in.  Every unit's sums go to a place of their
// own in the shared memory of the CTA that owns the tile; behind one cluster
// barrier the owners add them up in order.  (Measured instead: sums read from the
// others' shared memory behind the barrier cost 0.5 us a CTA of the cluster.)
// SMALL: INT4 codes as subnormal operands (bf16 results).
template <int FMT, int NT, bool SMALL>
__global__ void __launch_bounds__(Shape<NT>::kThreads, Shape<NT>::kCtas) k_gemv(Params P) {
  using S = Shape<NT>;
  constexpr bool INT4 = FMT == KQ_FMT_INT4_SYM || FMT == KQ_FMT_INT4_ASYM;
  constexpr bool BLOCKS = kByBlock<FMT, NT>;
  constexpr bool SUMS = FMT == KQ_FMT_INT4_ASYM || (FMT == KQ_FMT_INT4_SYM && SMALL);
  constexpr int kWarps = S::kWarps, kStep = S::kStep, kStages = S::kStages;
  extern __shared__ __align__(128) uint8_t smem[];
  // (what lies behind it is read by plain loads: a read-only load has no order with it)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int ranks = P.ranks, rank = ranks > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * (kStages * S::kStage);
  uint4* xs = reinterpret_cast<uint4*>(smem + kWarps * kStages * S::kStage);
  float2* xf = reinterpret_cast<float2*>(xs + P.seg * NT * 128);
  float* red = reinterpret_cast<float*>(xf + P.seg * NT * 8);
  // the others' shared memory may be written once they have all started
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  bool started = ranks == 1;
  const int64_t first_row = (int64_t)(blockIdx.x >> P.rank_shift) * P.tiles * 16;
  const int all_tiles = (int)min((int64_t)P.tiles, (P.n - first_row + 15) >> 4);
  const int own = (P.round + ranks - 1) >> P.rank_shift;  // tiles of a round a CTA owns at most
  const int mt = P.m, parts = P.parts;
  const int gbegin = rank_begin<NT>(P, rank), gend = rank_begin<NT>(P, rank + 1);
  // rounds: as many tiles as the sums have room for
  for (int t0 = 0; t0 < all_tiles; t0 += P.round) {
    const int tiles = min(P.round, all_tiles - t0);
    const int64_t row0 = first_row + 16 * (int64_t)t0;
    for (int g0 = gbegin; g0 < gend; g0 += P.seg) {
      // x stays staged from round to round where it is in one piece
      const bool fresh = t0 == 0 || gend - gbegin > P.seg;
      const int ng = min(P.seg, gend - g0), steps = (ng + kStep - 1) / kStep;
      // a warp's units: every kWarps-th (tile, part); a part is P.part steps
      struct Unit {
        int tile, part;
      };
      const Unit begin{warp >> P.part_shift, warp & (parts - 1)};
      auto next = [&](Unit& u) {
        u.tile += kWarps >> P.part_shift;
        u.part += kWarps & (parts - 1);
        if (u.part >= parts) {
          u.part -= parts;
          ++u.tile;
        }
      };
      Unit fu = begin;                      // copied next
      int fstep = 0, fend = 0, fill = 0;
      Stream<FMT, NT> stream;
      auto open = [&] {
        for (; fu.tile < tiles; next(fu)) {
          fstep = fu.part * P.part;
          fend = min(fstep + P.part, steps);
          if (fstep < fend) {
            stream.start(P, row0 + 16 * fu.tile);
            return;
          }
        }
      };
      auto fetch = [&] {
        if (fu.tile < tiles) {
          stream.copy(P, g0 + fstep * kStep, g0 + ng, ring + fill * S::kStage);
          if (++fill == kStages) fill = 0;
          if (++fstep == fend) {
            next(fu);
            open();
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      Eight x0{};
      if (fresh) x0 = load_x<NT>(P, g0, ng, 0);
      open();
#pragma unroll 1
      for (int i = 0; i < kStages; ++i) fetch();
      if (fresh) {
        if (t0 > 0 || g0 > gbegin) __syncthreads();   // the last segment's x is no longer read
        stage_x<SMALL, SUMS, BLOCKS, INT4, NT>(P, g0, ng, x0, xs, xf);
        __syncthreads();
      }
      if (!started) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
      started = true;
      int stage = 0;
#pragma unroll 1
      for (Unit u = begin; u.tile < tiles; next(u)) {
        const int tile = u.tile, part = u.part;
        const int s0 = part * P.part, s1 = min(s0 + P.part, steps);
        float acc[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
#pragma unroll 1
        for (int step = s0; step < s1; ++step) {
          asm volatile("cp.async.wait_group %0;" :: "n"(kStages - 1) : "memory");
          __syncwarp();
          compute_step<FMT, NT, SMALL>(ring + stage * S::kStage, step * kStep, ng - step * kStep, xs, xf, acc);
          __syncwarp();                     // the stage is free
          if (++stage == kStages) stage = 0;
          fetch();
        }
        const int owner = tile & (ranks - 1);
        float* to = red + (((rank * parts + part) * own + (tile >> P.rank_shift)) * 16 + g) * mt;
        if (owner != rank) to = cg::this_cluster().map_shared_rank(to, owner);
        // Two tokens a store where their number is even: 4-byte ones to other CTAs took a
        // seventh of 4096 x 2048 by 16 tokens.  (Four, by trading halves between lanes,
        // took as long as two.)
        if (g0 == gbegin && P.x_bf16 && (mt & 1) == 0) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const int tok = 8 * n + 2 * t;
            if (tok < mt) {
              *reinterpret_cast<float2*>(to + tok) = make_float2(acc[n][0], acc[n][1]);
              *reinterpret_cast<float2*>(to + 8 * mt + tok) = make_float2(acc[n][2], acc[n][3]);
            }
          }
        } else if (NT == 4 && gend - gbegin <= P.seg && !P.x_bf16 && (mt & 1) == 0) {
          // lanes t and t ^ 1 trade: the even one keeps row g, the odd one row g + 8
          const int odd = t & 1;
          float* half = to + (odd ? 8 * mt : 0);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float v0 = acc[n][0] + acc[n][1], v1 = acc[n][2] + acc[n][3];
            const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
            const int tok = 4 * n + (t & 2);
            if (tok < mt)
              *reinterpret_cast<float2*>(half + tok) = odd ? make_float2(other, v1)
                                                           : make_float2(v0, other);
          }
        } else {
          // behind the first segment: on top of what the same lane put there
          auto put = [&](float* at, float v) { *at = g0 > gbegin ? *at + v : v; };
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            if (P.x_bf16) {
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tok = 8 * n + 2 * t + (e & 1);
                if (tok < mt) put(to + 8 * (e >> 1) * mt + tok, acc[n][e]);
              }
            } else {
              const int tok = 4 * n + t;
              if (tok < mt) {
                put(to + tok, acc[n][0] + acc[n][1]);
                put(to + 8 * mt + tok, acc[n][2] + acc[n][3]);
              }
            }
          }
        }
      }
    }
    auto meet = [&] {
      if (ranks > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
      } else {
        __syncthreads();
      }
    };
    meet();
    // ---- join: the ranks' and parts' sums in order; a warp takes a tile by two tokens,
    // a lane a row
    const int mine = (tiles - rank + ranks - 1) >> P.rank_shift;    // tiles this CTA owns
    const int pairs = (mt + 1) >> 1, slots = ranks * parts, pitch = own * 16 * mt;
    const float t_scale = FMT == KQ_FMT_NVFP4 ? *P.tscale : 1.0f;
    for (int q = warp; q < mine * pairs; q += kWarps) {
      const int tl = q / pairs, tok = 2 * (q - tl * pairs) + (lane >> 4), r = lane & 15;
      const int64_t row = row0 + ((tl << P.rank_shift) + rank) * 16 + r;
      if (tok >= mt || row >= P.n) continue;
      const float* from = red + (tl * 16 + r) * mt + tok;
      float v = 0.0f;
#pragma unroll 8
      for (int c = 0; c < slots; ++c) v += from[c * pitch];
      if (SMALL) v *= 0x1p24f;              // the codes' 2^-24
      if (FMT == KQ_FMT_INT4_SYM) v *= static_cast<const float*>(P.scales)[row];
      if (FMT == KQ_FMT_NVFP4) v *= t_scale;
      const int64_t at = tok * P.n + row;
      if (P.y_bf16)
        static_cast<__nv_bfloat16*>(P.y)[at] = __float2bfloat16_rn(v);
      else
        static_cast<float*>(P.y)[at] = v;
    }
    if (t0 + P.round < all_tiles) meet();   // the sums are read: the next round's may come
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// What a CTA's work costs, in instructions of a warp (of two CTAs on an SM, its half):
// a step of a tile, a turn of staging x, a cluster's barriers, a further round of tiles.
// The number of CTAs that split k is the one with the least sum.  Measured, bf16 tokens,
// one rank against two: 1024 x 1024 by 1 token 3.2 and 3.5 us (one turn of staging
// either way), by 8 tokens 4.6 and 4.1; 32000 x 1536 by 8 tokens 11.5 and 13.2 (three
// steps are not halved).  Two against four: 4096 x 2048 by 16 tokens 8.0 and 7.5, 32000 x
// 2048 19.9 and 29.5 (two rounds and four; one rank, one round: 18.1).  8 ranks, which
// took the 4096 x 4096 product of one token from 6.3 to 6.6 us and the 12288 x 4096 one
// of eight from 11.8 to 13.3, only where x has no room otherwise.
template <int NT>
struct Cost {
  static constexpr int kStep = Shape<NT>::kStep * (60 + 40 * NT);
  static constexpr int kTurn = Shape<NT>::kWarps * 90, kTurnF32 = Shape<NT>::kWarps * 150;
  static constexpr int kBarrier = 1300 / Shape<NT>::kCtas;
  static constexpr int kRound = 13000 / Shape<NT>::kCtas;
};

// Shared memory of a CTA: the stages, x of a segment, the sums.
template <int NT>
struct Room {
  using S = Shape<NT>;
  static constexpr int kAll = (S::kCtas == 1 ? 227 : 113) * 1024;
  static constexpr int kRings = S::kWarps * S::kStages * S::kStage;
  static constexpr int kSums = (NT == 1 ? 12 : 20) * 1024;
  static constexpr int kGroups = (kAll - kRings - kSums) / (NT * (2048 + 64)) / S::kStep * S::kStep;
  static_assert(kGroups >= 4, "room for x");
};

// CTAs of clusters of `ranks` that the current device holds at a time: a cluster
// stays within a GPC, so it is less than all SMs hold.  Looked up once.
template <int FMT, int NT, bool SMALL>
cudaError_t resident_ctas(int ranks, int* out) {
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int i = ranks == 1 ? 0 : ranks == 2 ? 1 : ranks == 4 ? 2 : 3;
  if (dev < kDevices && (*out = known[dev][i].load(std::memory_order_relaxed)) > 0)
    return cudaSuccess;
  const size_t smem = Room<NT>::kAll;
  e = cudaFuncSetAttribute((const void*)k_gemv<FMT, NT, SMALL>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ranks);
  cfg.blockDim = dim3(Shape<NT>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  e = cudaOccupancyMaxActiveClusters(&clusters, (const void*)k_gemv<FMT, NT, SMALL>, &cfg);
  if (e != cudaSuccess) return e;
  if (clusters < 1) return cudaErrorInvalidConfiguration;   // none fits beside what is set aside
  *out = clusters * ranks;
  if (dev < kDevices) known[dev][i].store(*out, std::memory_order_relaxed);
  return cudaSuccess;
}

template <int FMT, int NT, bool SMALL>
cudaError_t launch(Params P, cudaStream_t s) {
  using R = Room<NT>;
  constexpr int kStep = Shape<NT>::kStep;
  const int64_t all = (P.n + 15) / 16;
  const int steps_all = (P.groups + kStep - 1) / kStep;
  auto groups_of = [&](int ranks) { return (steps_all + ranks - 1) / ranks * kStep; };
  const int room = R::kSums / (P.m * 64);               // tiles times parts, and a rank's rounding
  int ranks = 0;
  int64_t tiles = 0, least = 0;
  for (int r = 1; r <= 8; r *= 2) {
    if (r > 1 && P.groups < r * kStep) break;
    if (r < 8 ? groups_of(r) > R::kGroups : ranks > 0) continue;
    int ctas = 0;
    const cudaError_t e = resident_ctas<FMT, NT, SMALL>(r, &ctas);
    if (e != cudaSuccess) return e;
    // rows for as many clusters as run at a time
    const int clusters = ctas / r;
    const int64_t t = (all + clusters - 1) / clusters, rounds = (t + room - r) / (room - r + 1);
    const int64_t turns = (P.m * groups_of(r) + Shape<NT>::kThreads / 16 - 1) /
                          (Shape<NT>::kThreads / 16);
    const int64_t cost = t * (groups_of(r) / kStep) * Cost<NT>::kStep +
                         turns * (P.x_bf16 ? Cost<NT>::kTurn : Cost<NT>::kTurnF32) +
                         (r > 1 ? Cost<NT>::kBarrier : 0) + (rounds - 1) * Cost<NT>::kRound;
    if (ranks == 0 || cost < least) {
      ranks = r;
      tiles = t;
      least = cost;
    }
  }
  P.ranks = ranks;
  for (P.rank_shift = 0; 1 << P.rank_shift < ranks;) ++P.rank_shift;
  // x of a CTA's groups in one piece where there is room
  P.seg = groups_of(ranks);
  if (P.seg > R::kGroups) P.seg = R::kGroups;
  P.recip = (65536u + P.m - 1) / P.m;
  // a step's scales of a row are one or two aligned copies where every row begins at a
  // multiple of kStep groups
  const uintptr_t at = reinterpret_cast<uintptr_t>(P.scales) | reinterpret_cast<uintptr_t>(P.zeros);
  P.wide = P.groups % kStep == 0 && P.k % 128 == 0 &&
           at % (FMT == KQ_FMT_INT4_ASYM ? 2 * kStep : FMT == KQ_FMT_NVFP4 ? 16 : 4 * kStep) == 0;
  // in rounds as far as the sums fit
  P.tiles = (int)tiles;
  P.round = P.tiles;
  if (P.round > room - ranks + 1) {
    const int rounds = (P.tiles + room - ranks) / (room - ranks + 1);
    P.round = (P.tiles + rounds - 1) / rounds;
  }
  // parts: the shortest way through the units for the CTA's warps
  const int steps = P.seg / kStep, own = (P.round + ranks - 1) / ranks;
  int best = 1 << 30;
  for (int shift = 0, p = 1; (shift == 0 || p <= steps) && p * own * ranks <= room; ++shift, p *= 2) {
    const int turns = (P.round * p + Shape<NT>::kWarps - 1) / Shape<NT>::kWarps;
    const int part = (steps + p - 1) / p, way = turns * part;
    if (way < best) {
      best = way;
      P.parts = p;
      P.part_shift = shift;
      P.part = part;
    }
  }
  const size_t smem = R::kRings + (size_t)P.seg * NT * (2048 + 64) +
                      sizeof(float) * ranks * P.parts * own * 16 * P.m;
  if (smem > (size_t)R::kAll) return cudaErrorInvalidConfiguration;
  const cudaError_t e =
      cudaFuncSetAttribute((const void*)k_gemv<FMT, NT, SMALL>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, R::kAll);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)ranks;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  const cudaLaunchConfig_t cfg =
      dependent_launch(dim3((unsigned)((all + P.tiles - 1) / P.tiles * ranks)),
                       Shape<NT>::kThreads, smem, s, attr, ranks > 1 ? 1 : 0);
  return cudaLaunchKernelEx(&cfg, k_gemv<FMT, NT, SMALL>, P);
}

template <int FMT, bool SMALL>
cudaError_t launch_tiles(const Params& P, cudaStream_t s) {
  const int cols = P.x_bf16 ? P.m : 2 * P.m;
  if (cols <= 8) return launch<FMT, 1, SMALL>(P, s);
  if (cols <= 16) return launch<FMT, 2, SMALL>(P, s);
  return launch<FMT, 4, SMALL>(P, s);
}

}  // namespace gv

cudaError_t launch_gemv(int fmt, const void* x, int x_bf16, int m, const uint8_t* codes,
                        const void* scales, const void* zeros, const float* tscale, int64_t n,
                        int k, void* y, int y_bf16, cudaStream_t s) {
  const gv::Params P{x, codes, scales, static_cast<const uint16_t*>(zeros), tscale, y, n, m, k,
                     (k + 127) / 128, x_bf16, y_bf16, 0, 0, 0, 1, 0, 0, 1, 0, 0, 0};
  switch (fmt) {
    case KQ_FMT_INT4_SYM:
      return y_bf16 ? gv::launch_tiles<KQ_FMT_INT4_SYM, true>(P, s)
                    : gv::launch_tiles<KQ_FMT_INT4_SYM, false>(P, s);
    case KQ_FMT_INT4_ASYM:
      return y_bf16 ? gv::launch_tiles<KQ_FMT_INT4_ASYM, true>(P, s)
                    : gv::launch_tiles<KQ_FMT_INT4_ASYM, false>(P, s);
    case KQ_FMT_NVFP4: return gv::launch_tiles<KQ_FMT_NVFP4, false>(P, s);
    default: return gv::launch_tiles<KQ_FMT_MXFP4, false>(P, s);
  }
}

}  // namespace kq
