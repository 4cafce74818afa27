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

#include <atomic>
#include <cstdint>

#include "kq.h"
#include "kq_internal.h"
#include "kq_sm100.cuh"

namespace kq {
namespace gv {

namespace cg = cooperative_groups;
using sm100::pow2f;

// Up to two tiles of 8 columns: two CTAs of 8 warps an SM and units of 4 groups.
// Four tiles: one CTA of 16 warps, which stages x once an SM, and units of 2
// groups, so that two of them fit the registers beside the sums.
template <int NT>
struct Shape {
  static constexpr int kWarps = NT == 4 ? 16 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kCtas = NT == 4 ? 1 : 2;
  static constexpr int kBatch = NT == 4 ? 2 : 4;
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
  int tiles;                              // 16-row tiles of a cluster
  int seg;                                // groups whose x is staged at a time
  int parts;                              // batches of a CTA: sums kept apart
  int ranks, rank_shift;                  // CTAs of a cluster, which split k: 2^rank_shift
  int wide;                               // scales of kBatch groups in one load
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
__device__ __forceinline__ float half_value(uint32_t h) {
  return __half2float(__ushort_as_half((unsigned short)h));
}

// Codes are read once: not kept in L1, whole lines fetched into L2.
__device__ __forceinline__ uint4 load_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::128B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float2 half2_floats(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
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
    e.a = __ldg(p);
    if (!P.x_bf16) e.b = __ldg(p + 1);
  }
  return e;
}

// Stages x of groups [g0, g0 + ng) for the columns of NT mma tiles.  16 lanes take
// one (group, token), a lane 8 consecutive elements, which are one 16-byte piece
// in fragment order: (group, tile, word j, column, t) holds elements 32 t + 8 j ...
// as pairs (0,4) (1,5) (2,6) (3,7) for the masked INT4 codes, whose odd ones
// carry a factor 16, or in their own order for the converted E2M1 codes.  Columns
// behind the last one are left as they are: what they hold reaches no other
// column, and their sums are not stored.
template <bool INT4, int NT>
__device__ __forceinline__ void stage_x(const Params& P, int g0, int ng, uint4* xs, float2* xf) {
  constexpr int kAhead = 4;
  const int lane16 = threadIdx.x & 15, slot = threadIdx.x >> 4;
  const int items = ng * P.m;
  constexpr int kThreads = Shape<NT>::kThreads;
  for (int i0 = slot; i0 < items + slot; i0 += kAhead * (kThreads / 16)) {
    Eight in[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * (kThreads / 16), gi = i / P.m, tok = i - gi * P.m;
      in[u] = load8(P, i < items ? tok : P.m, (g0 + gi) * 128 + 8 * lane16);
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int i = i0 + u * (kThreads / 16), gi = i / P.m, tok = i - gi * P.m;
      if (__all_sync(0xffffffffu, i >= items)) break;
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
      const int sh = top > 0.0f ? min(141 - (int)(__float_as_uint(top) >> 23), 126) : 0;
      const float up = pow2f(sh);
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] *= up;
        sum += v[e];
      }
      if (INT4) {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      }
      if (i < items) {
        const int t = lane16 >> 2, j = lane16 & 3;
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          if (part == 1 && P.x_bf16) break;
          const int col = P.x_bf16 ? tok : 2 * tok + part;
          uint32_t h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float& lo = v[INT4 ? e : 2 * e];
            float& hi = v[INT4 ? e + 4 : 2 * e + 1];
            h[e] = half2_bits(lo, hi);
            if (!P.x_bf16 && part == 0) {
              const float2 r = half2_floats(h[e]);
              lo = (lo - r.x) * 2048.0f;
              hi = (hi - r.y) * 2048.0f;
            }
            if (INT4 && (e & 1)) h[e] = mul_h2(h[e], 0x2c002c00u);    // / 16
          }
          xs[((gi * NT + (col >> 3)) * 4 + j) * 32 + (col & 7) * 4 + t] =
              make_uint4(h[0], h[1], h[2], h[3]);
          // the sum of the group (of both parts at once) rides on the first column
          if (lane16 == 0)
            xf[gi * NT * 8 + col] = part == 0 ? make_float2(pow2f(-sh), sum * 0x1p-24f)
                                              : make_float2(pow2f(-sh) * 0x1p-11f, 0.0f);
        }
      }
    }
  }
}

// First group of a rank (ranks is a power of two).
__device__ __forceinline__ int rank_begin(const Params& P, int rank) {
  return (int)((uint32_t)(rank * P.groups) >> P.rank_shift);
}

// A unit of work as loaded: 16 rows (g and g + 8 of a lane) by kBatch groups.
template <int FMT, int kBatch>
struct Unit {
  uint4 a[kBatch], b[kBatch];
  uint32_t sa[kBatch], sb[kBatch];        // fp16 scale | zero << 16; E4M3 pair; E8M0 byte
};
template <int FMT, int kBatch>
__device__ __forceinline__ void load_unit(const Params& P, int64_t row0, int g0, int gend,
                                          Unit<FMT, kBatch>& u) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t last = P.n - 1;
  const int64_t ra = min(row0 + g, last), rb = min(row0 + 8 + g, last);
  const uint8_t* ca = P.codes + ra * (P.k / 2) + 16 * t + (int64_t)g0 * 64;
  const uint8_t* cb = P.codes + rb * (P.k / 2) + 16 * t + (int64_t)g0 * 64;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int gi = g0 + i;
    u.a[i] = u.b[i] = make_uint4(0, 0, 0, 0);
    if (gi < gend && gi * 128 + 32 * t < P.k) {
      u.a[i] = load_codes(ca + i * 64);
      u.b[i] = load_codes(cb + i * 64);
    }
  }
  if (P.wide && FMT == KQ_FMT_INT4_ASYM) {
    const uint16_t* s16 = static_cast<const uint16_t*>(P.scales) + g0;
    const uint16_t* z16 = P.zeros + g0;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t at = (r ? rb : ra) * P.groups;
      uint32_t* to = r ? u.sb : u.sa;
      uint32_t sw[kBatch / 2], zw[kBatch / 2];
      if constexpr (kBatch == 4) {
        const uint2 a = __ldg(reinterpret_cast<const uint2*>(s16 + at));
        const uint2 b = __ldg(reinterpret_cast<const uint2*>(z16 + at));
        sw[0] = a.x;
        sw[1] = a.y;
        zw[0] = b.x;
        zw[1] = b.y;
      } else {
        sw[0] = __ldg(reinterpret_cast<const uint32_t*>(s16 + at));
        zw[0] = __ldg(reinterpret_cast<const uint32_t*>(z16 + at));
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        to[i] = __byte_perm(sw[i / 2], zw[i / 2], i & 1 ? 0x7632 : 0x5410);
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int gi = g0 + i;
    u.sa[i] = u.sb[i] = 0;
    if (gi < gend && gi * 128 + 32 * t < P.k) {
      if (FMT == KQ_FMT_INT4_ASYM) {
        const uint16_t* s16 = static_cast<const uint16_t*>(P.scales) + gi;
        const uint16_t* z16 = P.zeros + gi;
        u.sa[i] = __ldg(s16 + ra * P.groups) | (uint32_t)__ldg(z16 + ra * P.groups) << 16;
        u.sb[i] = __ldg(s16 + rb * P.groups) | (uint32_t)__ldg(z16 + rb * P.groups) << 16;
      } else if (FMT == KQ_FMT_NVFP4) {
        const uint16_t* s16 = static_cast<const uint16_t*>(P.scales) + gi * 4 + t;
        u.sa[i] = __ldg(s16 + ra * (P.k / 32));
        u.sb[i] = __ldg(s16 + rb * (P.k / 32));
      } else if (FMT == KQ_FMT_MXFP4) {
        const uint8_t* s8 = static_cast<const uint8_t*>(P.scales) + gi * 4 + t;
        u.sa[i] = __ldg(s8 + ra * (P.k / 32));
        u.sb[i] = __ldg(s8 + rb * (P.k / 32));
      }
    }
  }
}

template <int FMT, int NT, int kBatch>
__device__ __forceinline__ void compute_unit(const Params& P, const Unit<FMT, kBatch>& u, int gl0, int ng,
                                             const uint4* xs, const float2* xf,
                                             float (&acc)[NT][4]) {
  constexpr bool INT4 = FMT == KQ_FMT_INT4_SYM || FMT == KQ_FMT_INT4_ASYM;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[n][j] = 0.0f;
#pragma unroll
  for (int i = 0; i < kBatch; ++i) {
    const int gl = gl0 + i;               // group within the staged segment
    if (gl >= ng) break;
    float c[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) c[n][j] = 0.0f;
    const uint32_t xa[4] = {u.a[i].x, u.a[i].y, u.a[i].z, u.a[i].w};
    const uint32_t xb[4] = {u.b[i].x, u.b[i].y, u.b[i].z, u.b[i].w};
    uint32_t ea = 0, eb = 0;              // MXFP4: largest exponent byte of the row's blocks
    uint32_t ma[2] = {0, 0}, mb[2] = {0, 0};
    if (FMT == KQ_FMT_NVFP4) {
      // both blocks' E4M3 scales as fp16, each in both halves
      uint32_t ha, hb;
      asm("{.reg .b16 v; cvt.u16.u32 v, %1; cvt.rn.f16x2.e4m3x2 %0, v;}" : "=r"(ha) : "r"(u.sa[i]));
      asm("{.reg .b16 v; cvt.u16.u32 v, %1; cvt.rn.f16x2.e4m3x2 %0, v;}" : "=r"(hb) : "r"(u.sb[i]));
      ma[0] = __byte_perm(ha, 0, 0x1010);
      ma[1] = __byte_perm(ha, 0, 0x3232);
      mb[0] = __byte_perm(hb, 0, 0x1010);
      mb[1] = __byte_perm(hb, 0, 0x3232);
    } else if (FMT == KQ_FMT_MXFP4) {
      ea = max(u.sa[i], __shfl_xor_sync(0xffffffffu, u.sa[i], 1));
      ea = max(ea, __shfl_xor_sync(0xffffffffu, ea, 2));
      eb = max(u.sb[i], __shfl_xor_sync(0xffffffffu, u.sb[i], 1));
      eb = max(eb, __shfl_xor_sync(0xffffffffu, eb, 2));
      auto down = [](uint32_t d) {        // 2^-d in both halves
        const uint32_t h = d < 15 ? (15 - d) << 10 : d < 25 ? 1u << (24 - d) : 0u;
        return h | h << 16;
      };
      ma[0] = ma[1] = down(ea - u.sa[i]);
      mb[0] = mb[1] = down(eb - u.sb[i]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t fa[4], fb[4];
      if (INT4) {
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
        const uint4 b = xs[((gl * NT + n) * 4 + j) * 32 + lane];
        mma16816(c[n], fa[0], fb[0], fa[1], fb[1], b.x, b.y);
        mma16816(c[n], fa[2], fb[2], fa[3], fb[3], b.z, b.w);
      }
    }
    // ---- the group's sums, scaled and added in fp32
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const float4 f4 = *reinterpret_cast<const float4*>(xf + gl * NT * 8 + 8 * n + 2 * t);
      const float2 f[2] = {make_float2(f4.x, f4.y), make_float2(f4.z, f4.w)};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 q = f[e & 1];
        const uint32_t s = e < 2 ? u.sa[i] : u.sb[i];
        if (FMT == KQ_FMT_INT4_ASYM)
          acc[n][e] = fmaf(half_value(s & 0xffffu) * q.x,
                           fmaf(-half_value(s >> 16), q.y, c[n][e]), acc[n][e]);
        else if (FMT == KQ_FMT_INT4_SYM)
          acc[n][e] = fmaf(q.x, fmaf(-8.0f, q.y, c[n][e]), acc[n][e]);
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

// A cluster takes 16 P.tiles rows and all of k, a CTA of it a range of k.  x of
// that range is staged once (in segments where k is long), while the first
// units' codes are on their way; then the warps take units, the next one's codes
// loaded before this one is computed.  Every unit's sums go to a place of their
// own in the shared memory of the CTA that owns the tile; behind one cluster
// barrier the owners add them up in order.  (Measured instead: sums read from the
// others' shared memory behind the barrier cost 0.5 us a CTA of the cluster.)
template <int FMT, int NT>
__global__ void __launch_bounds__(Shape<NT>::kThreads, Shape<NT>::kCtas) k_gemv(Params P) {
  constexpr bool INT4 = FMT == KQ_FMT_INT4_SYM || FMT == KQ_FMT_INT4_ASYM;
  constexpr int kBatch = Shape<NT>::kBatch, kWarps = Shape<NT>::kWarps;
  extern __shared__ __align__(16) uint8_t smem[];
  const int ranks = P.ranks, rank = ranks > 1 ? (int)cg::this_cluster().block_rank() : 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint4* xs = reinterpret_cast<uint4*>(smem);
  float2* xf = reinterpret_cast<float2*>(smem + (size_t)P.seg * NT * 2048);
  float* red = reinterpret_cast<float*>(xf + P.seg * NT * 8);
  // the others' shared memory may be written once they have all started
  if (ranks > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  bool started = ranks == 1;
  const int64_t row0 = (int64_t)(blockIdx.x >> P.rank_shift) * P.tiles * 16;
  const int tiles = (int)min((int64_t)P.tiles, (P.n - row0 + 15) >> 4);
  const int own = (P.tiles + ranks - 1) >> P.rank_shift;  // tiles a CTA owns at most
  const int mt = P.m;
  const int gbegin = rank_begin(P, rank), gend = rank_begin(P, rank + 1);
  for (int g0 = gbegin; g0 < gend; g0 += P.seg) {
    const int ng = min(P.seg, gend - g0), first_part = (g0 - gbegin) / kBatch;
    const int parts = (ng + kBatch - 1) / kBatch, units = tiles * parts;
    Unit<FMT, kBatch> u;
    auto load = [&](int i) {
      const int tile = i / parts, part = i - tile * parts;
      load_unit<FMT, kBatch>(P, row0 + 16 * tile, g0 + part * kBatch, g0 + ng, u);
    };
    int i = warp;
    if (i < units) load(i);
    if (g0 > gbegin) __syncthreads();     // the last segment's x is no longer read
    stage_x<INT4, NT>(P, g0, ng, xs, xf);
    __syncthreads();
    if (!started) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
    started = true;
    for (; i < units; i += kWarps) {
      const int tile = i / parts, part = i - tile * parts;
      const Unit<FMT, kBatch> now = u;
      if (i + kWarps < units) load(i + kWarps);
      float acc[NT][4];
      compute_unit<FMT, NT, kBatch>(P, now, part * kBatch, ng, xs, xf, acc);
      const int owner = tile & (ranks - 1);
      float* to = red + (size_t)(((rank * P.parts + first_part + part) * own + (tile >> P.rank_shift)) * 16 +
                                 g) * mt;
      if (owner != rank) to = cg::this_cluster().map_shared_rank(to, owner);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        if (P.x_bf16) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = 8 * n + 2 * t + (e & 1);
            if (tok < mt) to[8 * (e >> 1) * mt + tok] = acc[n][e];
          }
        } else {
          const int tok = 4 * n + t;
          if (tok < mt) {
            to[tok] = acc[n][0] + acc[n][1];
            to[8 * mt + tok] = acc[n][2] + acc[n][3];
          }
        }
      }
    }
  }
  if (ranks > 1) {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  } else {
    __syncthreads();
  }
  // ---- join: the ranks' batches in order; consecutive threads take consecutive
  // rows of one token
  const int mine = ((tiles - rank + ranks - 1) >> P.rank_shift) * 16;   // rows this CTA owns
  for (int i = threadIdx.x; i < mine * mt; i += Shape<NT>::kThreads) {
    const int tok = i / mine, r = i - tok * mine;
    const int64_t row = row0 + (int64_t)((r >> 4) * ranks + rank) * 16 + (r & 15);
    if (row >= P.n) continue;
    const float* from = red + (size_t)r * mt + tok;
    float v = 0.0f;
    for (int c = 0; c < ranks; ++c) {
      const int parts = (rank_begin(P, c + 1) - rank_begin(P, c) + kBatch - 1) / kBatch;
#pragma unroll 4
      for (int w = 0; w < parts; ++w) v += from[(size_t)(c * P.parts + w) * own * 16 * mt];
    }
    if (INT4) v *= 0x1p24f;               // the codes' 2^-24
    if (FMT == KQ_FMT_INT4_SYM) v *= static_cast<const float*>(P.scales)[row];
    if (FMT == KQ_FMT_NVFP4) v *= *P.tscale;
    const int64_t at = (int64_t)tok * P.n + row;
    if (P.y_bf16)
      static_cast<__nv_bfloat16*>(P.y)[at] = __float2bfloat16_rn(v);
    else
      static_cast<float*>(P.y)[at] = v;
  }
}

#ifndef KQ_RANKS
#define KQ_RANKS 4
#endif
constexpr size_t kMostX = 65536 + 2048, kMostSums = 32768;   // shared memory of a CTA

// CTAs of clusters of `ranks` that the current device holds at a time: a cluster
// stays within a GPC, so it is less than all SMs hold.  Looked up once.
template <int FMT, int NT>
cudaError_t resident_ctas(int ranks, int* out) {
  // the attribute set here holds for every launch of this kernel on the device
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices][4];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int i = ranks == 1 ? 0 : ranks == 2 ? 1 : ranks == 4 ? 2 : 3;
  if (dev < kDevices && (*out = known[dev][i].load(std::memory_order_relaxed)) > 0)
    return cudaSuccess;
  const size_t smem = Shape<NT>::kCtas == 1 ? 2 * kMostX + kMostSums : kMostX + kMostSums;
  e = cudaFuncSetAttribute((const void*)k_gemv<FMT, NT>,
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
  e = cudaOccupancyMaxActiveClusters(&clusters, (const void*)k_gemv<FMT, NT>, &cfg);
  if (e != cudaSuccess) return e;
  *out = clusters * ranks;
  if (dev < kDevices) known[dev][i].store(*out, std::memory_order_relaxed);
  return cudaSuccess;
}

template <int FMT, int NT>
cudaError_t launch(Params P, cudaStream_t s) {
  constexpr int kBatch = Shape<NT>::kBatch;
  int ranks = 1;
  while (ranks < KQ_RANKS && P.groups / (2 * ranks) >= kBatch) ranks *= 2;
  while (ranks < 8 && P.groups / ranks > 128) ranks *= 2;
  P.ranks = ranks;
  for (P.rank_shift = 0; 1 << P.rank_shift < ranks;) ++P.rank_shift;
  int ctas = 0;
  cudaError_t e = resident_ctas<FMT, NT>(ranks, &ctas);
  if (e != cudaSuccess) return e;
  const int64_t all = (P.n + 15) / 16;
  // x of a CTA's groups in one piece where 64 KB (128 KB for one CTA an SM) hold it
  const int mine = (P.groups + ranks - 1) / ranks;
  P.parts = (mine + kBatch - 1) / kBatch;
  P.seg = P.parts * kBatch;
  const int most = 131072 / Shape<NT>::kCtas / (2048 * NT);
  if (P.seg > most) P.seg = most;
  // the scales of kBatch groups are one aligned load where every range and row
  // begins at a multiple of kBatch groups
  P.wide = P.groups % (kBatch * ranks) == 0 &&
           (reinterpret_cast<uintptr_t>(P.scales) | reinterpret_cast<uintptr_t>(P.zeros)) %
                   (2 * kBatch) == 0;
  // rows for one round of CTAs, as far as their sums fit 32 KB
  int64_t tiles = (all + ctas / ranks - 1) / (ctas / ranks);
  const int64_t cap = kMostSums / ((int64_t)P.parts * P.m * 64);
  if (tiles > cap) tiles = cap;
  P.tiles = (int)(tiles < 1 ? 1 : tiles);
  const int own = (P.tiles + ranks - 1) / ranks;
  const size_t smem = (size_t)P.seg * NT * (2048 + 64) +
                      sizeof(float) * ranks * P.parts * own * 16 * P.m;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((all + P.tiles - 1) / P.tiles * ranks));
  cfg.blockDim = dim3(Shape<NT>::kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = ranks > 1 ? 1 : 0;
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
                     (k + 127) / 128, x_bf16, y_bf16, 0, 0, 0, 1, 0, 0};
  switch (fmt) {
    case KQ_FMT_INT4_SYM: return gv::launch_tiles<KQ_FMT_INT4_SYM>(P, s);
    case KQ_FMT_INT4_ASYM: return gv::launch_tiles<KQ_FMT_INT4_ASYM>(P, s);
    case KQ_FMT_NVFP4: return gv::launch_tiles<KQ_FMT_NVFP4>(P, s);
    default: return gv::launch_tiles<KQ_FMT_MXFP4>(P, s);
  }
}

}  // namespace kq
