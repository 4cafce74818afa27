// Attention of one new token per sequence over the paged INT4 KV cache that
// kq_rht_quant_int4_kv writes (QuaRot reviews, final comments: the KV cache at
// 4 bits with a per-head 128-point Hadamard).  Keys and values are stored
// rotated, so the query is rotated on the way in (q . k is unchanged when both
// carry the rotation) and the result rotated back on the way out.
//
// Mathematics.  With codes u, scales s and zero points z of a token's head,
//   a_t = f s_t (sum_d q_d u_td - z_t sum_d q_d),   p_t = 2^(a_t - max a)
//   o_d = (sum_t (p_t s'_t) u_td - sum_t (p_t s'_t) z'_t) / sum_t p_t
// so both products run on the bare 4-bit codes: bits masked out of their word
// ARE an fp16 number (a pattern below 2^11 means itself times 2^-24), exact on
// the tensor cores.  The operands are a byte, 16 h + l, and its low code l, which
// cost 4 integer operations per 8 codes; h is taken out of them in the query's
// coefficients (keys) and in the result (values).  The tensor core lines up such
// subnormal operands as if they were 2^-14, so terms keep 15 bits of the largest in
// their step (the query's and the weights' 11 bits cost more); sums are fp32.
//
// Bound by HBM: each visible token is read once, 68 bytes a head for the key
// and 68 for the value.  mma.sync (m16n8k16) carries the contraction: its 16
// rows are tokens (scores) or dimensions (values), its 8 columns the query
// heads that share the cached head, and at the memory's rate it needs 3/8 of
// that path's throughput; the accumulators stay where the softmax is computed.
// Measured (one B200, time between calls in a graph): one sequence of 131071
// tokens, 8 cached and 64 query heads, 42.7 us = 3.3 TB/s, of which 30 us are the
// tiles, 6 the start (lengths, pages and query, one memory latency behind the other)
// and 6 the join; 32 sequences of 300 to 4096 tokens 23.5 us.  In the tiles memory and
// instruction issue are near each other: without the copies they take 25 us, at 1.9
// to 2.0 instructions a cycle, half of them on the integer pipe (unpacking).
//
// Work split.  The visible tokens of all (sequence, head block, column chunk)
// units are cut into tiles, and the tiles dealt to the CTAs in contiguous
// ranges of equal length, computed on the device from seq_lens: long and short
// sequences load the machine alike and nothing depends on host knowledge of
// the lengths.  A unit that one CTA covers is finished there; the others leave
// partial sums in the workspace, and which CTAs they are, which a second small kernel
// (launched as a programmatic dependent) joins in CTA order.  (Measured instead: the
// join adding up the lengths again to find the CTAs, 1.2 to 1.6 us slower behind its
// wait; a cooperative launch that joins behind a barrier of the grid, 5 us slower in
// every case; the last CTA of a unit to arrive, 47.6 for 24.5 us.)  Few and short sequences, by what the
// table and the window allow, are not cut: a CTA takes a unit, and nothing is joined.
//
// Per CTA: eight warps compute, each its own head (or its own part of the tokens
// when there are fewer heads), and fill the shared stages together with 16-byte
// asynchronous copies, one barrier a tile.  (Measured instead: bulk copies issued
// lane by lane took 100 cycles each, 6500 a tile; extra warps for the copies
// left the others 96 registers, which spilled; one CTA of 16 warps an SM, two warps a
// head, rotated each query once an SM but waited at its barrier, 44.2 us.)  Stage rows
// are 32 bytes longer than a multiple of 128, which keeps both fragment reads free of bank conflicts.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>
#include <cstdint>

#include "kq_internal.h"
#include "kq_mma16.cuh"
#include "kq_sm100.cuh"

namespace kq {
namespace at {

using namespace sm100;

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
// A running maximum is kept until a score passes it by more than this (in
// powers of two); the weights stay below 2^kSlack.
constexpr int kSlack = 6;
constexpr int kCols = 8;                      // query heads a unit carries
constexpr int kMaxCtas = 320;
// What beginning a unit costs, in tiles: the query's rotation and the end of the
// unit before it.  The tiles are dealt with so many more in front of each unit.
constexpr int kUnitCost = 2;
// Where no sequence shows more tokens than this and every unit of one head finds a
// CTA at once, a CTA takes a unit: no lengths to add up, nothing to join, one launch.
// 4 sequences, 8 cached and 32 query heads, GPU time (time per call from the host),
// dealt or alone: 256 tokens 8.6 (9.8) or 7.5 (7.7) us, 512 9.2 (9.7) or 9.4 (9.4), 1024
// 11.3 (11.7) or 13.3 (13.3); 37 sequences of 512, 296 units, 14.8 or 13.5; 64 of 128, 512
// units, 13.0 or 16.6.
constexpr int kAloneTokens = 512;
constexpr int kPartFloats = kCols * 128 + 2 * kCols;   // o, m, l of one head
// The workspace: partial sums of [CTA][first unit, last unit][head], then of each unit
// the CTAs that worked on it.
constexpr size_t kPartBytes = sizeof(float) * kMaxCtas * 2 * kWarps * kPartFloats;
struct Span {
  int first;                // 2 CTA + place of its partial sums
  int last;                 // CTA
};
__device__ __forceinline__ Span* span_of(const AttnArgs& P, int64_t b, int blocks, int hb,
                                         int chunks, int chunk) {
  return reinterpret_cast<Span*>(static_cast<char*>(P.workspace) + kPartBytes) +
         ((b * blocks + hb) * chunks + chunk);
}

// Tokens of one sequence: positions v < vis, v + skip from `sinks` on.
struct Seq {
  int vis, skip;
};
__device__ __forceinline__ Seq sequence(const AttnArgs& P, int most, int64_t b) {
  const int len = min(max(P.seq_lens[b], 0), most);
  const int64_t keep = (int64_t)P.window + P.sinks;
  Seq s;
  s.skip = P.window > 0 && len > keep ? (int)(len - keep) : 0;
  s.vis = len - s.skip;
  return s;
}
__device__ __forceinline__ int longest(const AttnArgs& P) {
  const int64_t most = P.table_width * P.page_size;
  return most > 0x7fffffff ? 0x7fffffff : (int)most;
}

// How `total` tiles are dealt: `ctas` contiguous ranges, the first `more` of
// them one tile longer than `each`.
struct Deal {
  int64_t each;
  int ctas, more;
};
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
  // 32-bit division where it reaches (a 64-bit one costs several hundred cycles)
  return (a | b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}
__device__ __forceinline__ Deal deal(int64_t total, int grid) {
  Deal d;
  d.ctas = total < grid ? (int)total : grid;
  d.each = div64(total, d.ctas);
  d.more = (int)(total - d.each * d.ctas);
  return d;
}
__device__ __forceinline__ int64_t cta_first(const Deal& d, int c) {
  return c * d.each + min(c, d.more);
}

// A walk over a CTA's tiles: sequence, block of heads, chunk of query heads, tile;
// `left` tiles remain for the CTA (units still to begin cost kUnitCost of them).
struct Walk {
  int64_t b;
  int hb, chunk, tile, tiles, left;
  Seq seq;
};
template <int TILE>
__device__ __forceinline__ void step(const AttnArgs& P, int most, int blocks, int chunks, Walk& w) {
  --w.left;
  if (++w.tile < w.tiles) return;
  w.left -= kUnitCost;
  if (w.left <= 0) return;
  w.tile = 0;
  if (++w.chunk < chunks) return;
  w.chunk = 0;
  if (++w.hb < blocks) return;
  w.hb = 0;
  do {
    ++w.b;
    w.seq = sequence(P, most, w.b);
    w.tiles = (w.seq.vis + TILE - 1) / TILE;
  } while (w.tiles == 0);
}
// What a unit of sequence b0 + lane costs, in tiles (0 behind the last one and for
// an empty one), and the inclusive sum over the lanes (at most 2^26 a sequence).
template <int TILE>
__device__ __forceinline__ void scan32(const AttnArgs& P, int most, int64_t b0, Seq& seq,
                                       uint32_t& n, uint32_t& incl) {
  const int lane = threadIdx.x & 31;
  seq = Seq{0, 0};
  if (b0 + lane < P.batch) seq = sequence(P, most, b0 + lane);
  n = incl = seq.vis > 0 ? (uint32_t)(seq.vis + TILE - 1) / TILE + kUnitCost : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
}
// Deals the tiles and starts the CTA's walk; false when nothing is left for it.
template <int TILE>
__device__ __forceinline__ bool begin(const AttnArgs& P, int most, int blocks, int chunks, Walk& w) {
  Seq seq;
  uint32_t n, incl;
  const int subs = blocks * chunks;
  scan32<TILE>(P, most, 0, seq, n, incl);
  int64_t total = __shfl_sync(0xffffffffu, incl, 31);
  for (int64_t b0 = 32; b0 < P.batch; b0 += 32) {
    Seq other;
    uint32_t k, sum;
    scan32<TILE>(P, most, b0, other, k, sum);
    total += __shfl_sync(0xffffffffu, sum, 31);
  }
  total *= subs;
  if (total == 0) return false;
  const Deal dl = deal(total, gridDim.x);
  if ((int)blockIdx.x >= dl.ctas) return false;
  const int64_t first = cta_first(dl, blockIdx.x);
  w.left = (int)(cta_first(dl, blockIdx.x + 1) - first);
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < P.batch; b0 += 32) {
    if (b0 > 0) scan32<TILE>(P, most, b0, seq, n, incl);
    const unsigned hit = __ballot_sync(0xffffffffu, (base + incl) * subs > first);
    if (hit) {
      const int l = __ffs(hit) - 1;
      const int cost = (int)__shfl_sync(0xffffffffu, n, l);
      w.b = b0 + l;
      w.seq.vis = __shfl_sync(0xffffffffu, seq.vis, l);
      w.seq.skip = __shfl_sync(0xffffffffu, seq.skip, l);
      w.tiles = cost - kUnitCost;
      const int64_t before = base + __shfl_sync(0xffffffffu, incl, l) - cost;
      const int64_t off = first - before * subs;
      const int sub = (int)div64(off, cost);
      w.hb = sub / chunks;
      w.chunk = sub - w.hb * chunks;
      w.tile = (int)(off - (int64_t)sub * cost) - kUnitCost;
      if (w.tile < 0) {                  // the range begins in front of the unit
        w.left += w.tile;
        w.tile = 0;
      }
      return w.left > 0;
    }
    base += __shfl_sync(0xffffffffu, incl, 31);
  }
  return false;
}

// pos / page_size for pos < 2^31 by a multiplication (Granlund and Montgomery, Division by
// invariant integers using multiplication, 1994): with l = ceil(log2 d) and
// M = ceil(2^(31 + l) / d), M d - 2^(31 + l) < d <= 2^l, so floor(pos M / 2^(31 + l))
// is the quotient.  M = 0 stands for d = 1.
struct PageDiv {
  uint32_t mul, shift;
};
__device__ __forceinline__ uint32_t page_of(PageDiv d, uint32_t pos) {
  return d.mul ? __umulhi(pos, d.mul) >> d.shift : pos;
}
// Where visible token v lies: its page as the table has it (an asynchronous
// load whose value is looked at one tile later) and its place in the page.
struct Place {
  int page, in;
};
__device__ __forceinline__ Place place(const AttnArgs& P, PageDiv d, const Walk& w, int v) {
  if (v >= w.seq.vis) return Place{-1, 0};
  const uint32_t pos = (uint32_t)(v < P.sinks ? v : v + w.seq.skip);
  const uint32_t page_in = page_of(d, pos);
  return Place{P.block_table[w.b * P.table_width + page_in],
               (int)(pos - page_in * (uint32_t)P.page_size)};
}
// Its cache row, -1 where there is none.
__device__ __forceinline__ int cache_row(const AttnArgs& P, Place p) {
  const int64_t row = (int64_t)p.page * P.page_size + p.in;
  return p.page < 0 || row >= P.num_slots ? -1 : (int)row;
}

template <int HB>
struct Shape {
  static constexpr int kSplit = kWarps / HB;             // warps a head
  static constexpr int kTok = HB == 1 ? 16 : 32;         // tokens a warp and tile
  static constexpr int kTile = kTok * kSplit;            // tokens a tile
  static constexpr int kRow = HB * 64 + 32;              // bytes a staged code row
  static constexpr int kCodes = kTile * kRow;            // keys or values of a tile
  // [4][kTile][HB] halves: key scales and zero points, value scales and zero
  // points; then a byte a token: not visible
  static constexpr int kArray = kTile * HB * 2;
  static constexpr int kScales = 4 * kArray;
  static constexpr int kMask = kTile;
  static constexpr int kLanes = HB == 1 ? 4 : 8;         // lanes that copy a row
  static constexpr int kPass = 32 / kLanes;              // rows a warp copies at a time
  static constexpr int kPasses = kTile / kWarps / kPass;
  static constexpr int kStage = 2 * kCodes + kScales + kMask;
  static constexpr int kStages = HB == 8 ? 3 : HB == 1 ? 3 : 2;
  // the warps of a head are joined two by two: one writes, one adds
  static constexpr int kJoin = kSplit > 1 ? kWarps / 2 * kPartFloats * 4 : 0;
  static constexpr size_t kSmem = kStages * kStage + kJoin;
};

// 16 bytes, both addresses with a constant offset.
template <int OFFSET>
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %2], 16;"
               :: "r"(dst), "l"(src), "n"(OFFSET) : "memory");
}
// BYTES, or zeros (and no read).
template <int BYTES>
__device__ __forceinline__ void copy_or_zero(uint32_t dst, const void* src, bool in) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;"
                 :: "r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;"
                 :: "r"(dst), "l"(src), "n"(BYTES), "r"(in ? BYTES : 0) : "memory");
}
// Every 128th byte's 16 of a row of HB heads (64 bytes a head).
template <int HB>
__device__ __forceinline__ void copy_lines(uint32_t dst, const uint8_t* src) {
  copy16<0>(dst, src);
  if constexpr (HB > 2) copy16<128>(dst, src);
  if constexpr (HB > 4) {
    copy16<256>(dst, src);
    copy16<384>(dst, src);
  }
}
__device__ __forceinline__ void commit_copies() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void wait_copies() {   // at most N groups still under way
  asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}
__device__ __forceinline__ float exp2_(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_over_rows(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
}
__device__ __forceinline__ float sum_over_rows(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 4);
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  return v + __shfl_xor_sync(0xffffffffu, v, 16);
}
// 16 dimensions a lane (16 (lane / 4) + i): unnormalized H_128 over the 8 lanes.
__device__ __forceinline__ void hadamard_rows(float (&v)[16]) {
#pragma unroll
  for (int st = 1; st < 16; st <<= 1)
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!(i & st)) {
        const float a = v[i], b = v[i | st];
        v[i] = a + b;
        v[i | st] = a - b;
      }
#pragma unroll
  for (int st = 4; st < 32; st <<= 1) {
    const float own = (threadIdx.x & st) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = fmaf(own, v[i], __shfl_xor_sync(0xffffffffu, v[i], st));
  }
}
// Rotates 16 values a lane back, applies the signs and stores them as bf16.
__device__ __forceinline__ void store_result(const AttnArgs& P, float (&v)[16], int64_t b, int qh,
                                             int kh, bool store) {
  hadamard_rows(v);
  const int d0 = 16 * ((threadIdx.x & 31) >> 2);
  uint32_t w[8];
  uint4 sg = make_uint4(0, 0, 0, 0);
  if (P.v_signs) sg = *reinterpret_cast<const uint4*>(P.v_signs + kh * 128 + d0);
  const uint32_t s4[4] = {sg.x, sg.y, sg.z, sg.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float r[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int e = 2 * i + j;
      const uint32_t neg = s4[e >> 2] << (24 - 8 * (e & 3)) & 0x80000000u;
      r[j] = __uint_as_float(__float_as_uint(v[e] * 0.08838834764831845f) ^ neg);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(r[0], r[1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (store) {
    uint4* to = reinterpret_cast<uint4*>(static_cast<uint16_t*>(P.out) +
                                         (b * P.q_heads + qh) * 128 + d0);
    to[0] = make_uint4(w[0], w[1], w[2], w[3]);
    to[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// ALONE: a CTA takes one unit, from its first tile to its last.
template <int HB, bool ALONE>
__global__ void __launch_bounds__(kThreads, 2) k_attn(AttnArgs P, PageDiv pages) {
  using S = Shape<HB>;
  constexpr int TILE = S::kTile, MB = S::kTok / 16;
  extern __shared__ __align__(128) uint8_t smem[];
  float* join = reinterpret_cast<float*>(smem + S::kStages * S::kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the join, whose CTAs may come in as soon as this kernel's leave room
  if (!ALONE) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int most = longest(P);
  const int group = P.q_heads / P.kv_heads, chunks = (group + kCols - 1) / kCols;
  const int blocks = P.kv_heads / HB;
  Walk w;
  bool any;
  if constexpr (ALONE) {
    const int unit = blockIdx.x / chunks;
    w.chunk = blockIdx.x - unit * chunks;
    w.b = unit / blocks;
    w.hb = unit - (int)w.b * blocks;
    w.seq = sequence(P, most, w.b);
    w.tile = 0;
    w.left = w.tiles = (w.seq.vis + TILE - 1) / TILE;
    any = w.left > 0;
  } else {
    any = begin<TILE>(P, most, blocks, chunks, w);
  }
  // sequences without a visible token have no tile: their rows are zeros
  for (int64_t b = blockIdx.x; b < P.batch; b += gridDim.x)
    if (sequence(P, most, b).vis == 0)
      for (int i = threadIdx.x; i < P.q_heads * 16; i += kThreads)
        reinterpret_cast<uint4*>(P.out)[b * P.q_heads * 16 + i] = make_uint4(0, 0, 0, 0);
  if (!any) return;

  // ================= filling the stages.  A warp copies kTile / 8 rows, 8 lanes a
  // row (4 when a row is one head), a lane 16 bytes of each of the row's 128-byte
  // lines: the copies of a row differ by constants alone, and every request is a
  // whole line.  A token that is not visible gets the codes of row 0 (any codes
  // do: its weight is zero).  The first four lanes of a row also copy its scales
  // and zero points, an array each (2 bytes, where a row is one head, are too few
  // for an asynchronous copy and go through a register into the stage one tile
  // later).  Pages are looked up one tile ahead.
  const int arr = lane % S::kLanes;
  const uint16_t* sc_from = arr == 0 ? P.k_scales : arr == 1 ? P.k_zeros
                            : arr == 2 ? P.v_scales : P.v_zeros;
  const int my_row = warp * (TILE / kWarps) + lane / S::kLanes;    // + pass * kPass
  const uint32_t my_codes = smem_u32(smem) + (uint32_t)my_row * S::kRow + 16 * arr;
  const uint32_t my_scales = smem_u32(smem) + 2 * S::kCodes + arr * S::kArray + my_row * HB * 2;
  Walk ahead = w;
  int fill = 0;                           // stage to fill
  [[maybe_unused]] int late = -1;         // stage whose scales are still in registers
  [[maybe_unused]] uint16_t sreg[S::kPasses];
  Place at[S::kPasses];
  auto look = [&] {
#pragma unroll
    for (int j = 0; j < S::kPasses; ++j)
      at[j] = place(P, pages, ahead, ahead.tile * TILE + my_row + j * S::kPass);
  };
  auto store_scales = [&] {
    if constexpr (HB == 1) {
      if (late < 0) return;
#pragma unroll
      for (int j = 0; j < S::kPasses; ++j)
        *reinterpret_cast<uint16_t*>(smem + late * S::kStage + 2 * S::kCodes + arr * S::kArray +
                                     (my_row + j * S::kPass) * 2) = sreg[j];
      late = -1;
    }
  };
  auto fetch = [&] {
    if (ahead.left > 0) {
      const int head0 = ahead.hb * HB;
      const uint32_t base = fill * S::kStage;
#pragma unroll
      for (int j = 0; j < S::kPasses; ++j) {
        const int r = cache_row(P, at[j]);
        const int64_t row = (int64_t)max(r, 0) * P.kv_heads + head0;
        const int64_t off = row * 64 + 16 * arr;
        const uint32_t to = my_codes + base + j * S::kPass * S::kRow;
        copy_lines<HB>(to, P.k_codes + off);
        copy_lines<HB>(to + S::kCodes, P.v_codes + off);
        if constexpr (HB == 1) {
          sreg[j] = r >= 0 ? sc_from[row] : 0;
        } else {
          if (arr < 4)
            copy_or_zero<2 * HB>(my_scales + base + j * S::kPass * HB * 2, sc_from + row, r >= 0);
        }
        if (arr == 0) smem[base + 2 * S::kCodes + S::kScales + my_row + j * S::kPass] = r < 0;
      }
      late = fill;
      if (++fill == S::kStages) fill = 0;
      step<TILE>(P, most, blocks, chunks, ahead);
      if (ahead.left > 0) look();
    }
    commit_copies();
  };
  look();
#pragma unroll 1
  for (int i = 0; i + 1 < S::kStages; ++i) {
    store_scales();
    fetch();
  }

  int stage = 0;
  {
    // ================= compute: head `hw` of the block, tokens tok0 .. of a tile
    const int hw = warp / S::kSplit, part = warp % S::kSplit;
    const int tok0 = part * S::kTok;
    const int g = lane >> 2, t = lane & 3;
    // the tokens of accumulator rows 2t and 2t + 1, and of row g
    const int even = t, odd = 4 + ((t + 2) & 3);
    const int mine = g & 1 ? 4 + (((g >> 1) + 2) & 3) : g >> 1;
    uint32_t qf[4][4];
    float fa[2], fz[2];                    // per column 2t, 2t + 1
    float m[2], ref[2], l[2], zs[4], o[8][4];
    int ev = 0;
    // no visible token of the unit seen yet: a tile whose pages lie outside the cache
    // leaves m at -infinity, which would take the weights added behind it to zero
    bool fresh = false;
    int segment = 0;
    while (w.left > 0) {
      // ---- the unit's query, rotated; lane (g, t) holds dimensions 32 t .. of column g
      const int kh = w.hb * HB + hw;
      const int col0 = w.chunk * kCols;
      const int columns = min(kCols, group - col0);
      {
        float q[32];
        {
          const uint4* from = reinterpret_cast<const uint4*>(
              static_cast<const uint16_t*>(P.q) +
              (w.b * P.q_heads + (int64_t)kh * group + col0 + min(g, columns - 1)) * 128 + 32 * t);
          const uint4* sp = reinterpret_cast<const uint4*>(P.k_signs + kh * 128 + 32 * t);
          uint4 v[4], sg[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = from[i];
          if (P.k_signs) {
            sg[0] = sp[0];
            sg[1] = sp[1];
          }
          const uint32_t ok = g < columns ? 0xffffffffu : 0u;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint4 x4 = v[i >> 2], s4 = sg[i >> 3];
            const uint32_t x = (i & 3) == 0 ? x4.x : (i & 3) == 1 ? x4.y : (i & 3) == 2 ? x4.z : x4.w;
            const uint32_t c = (i >> 1 & 3) == 0 ? s4.x : (i >> 1 & 3) == 1 ? s4.y
                               : (i >> 1 & 3) == 2 ? s4.z : s4.w;
            // the sign bytes' top bits onto those of the two bf16 values
            const uint32_t flip = __byte_perm(c, 0, i & 1 ? 0x3424 : 0x1404) & 0x80008000u;
            const uint32_t y = (x ^ flip) & ok;
            q[2 * i] = __uint_as_float(y << 16);
            q[2 * i + 1] = __uint_as_float(y & 0xffff0000u);
          }
        }
#pragma unroll
        for (int st = 1; st < 32; st <<= 1)
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!(i & st)) {
              const float a = q[i], b = q[i | st];
              q[i] = a + b;
              q[i | st] = a - b;
            }
        float top = 0.0f;
#pragma unroll
        for (int st = 1; st < 4; st <<= 1) {
          const float own = (lane & st) ? -1.0f : 1.0f;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            q[i] = fmaf(own, q[i], __shfl_xor_sync(0xffffffffu, q[i], st));
        }
#pragma unroll
        for (int i = 0; i < 32; i += 2) top = fmax3(top, fabsf(q[i]), fabsf(q[i + 1]));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // fp16 with a power of two per column that puts its largest element in
        // [2^13, 2^14): 11 significant bits over 27 binades
        const int ex = (int)(__float_as_uint(top) >> 23) - 127;
        const int sh = top > 0.0f ? min(max(13 - ex, -120), 120) : 0;
        const float up = pow2f(sh);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // a byte 16 h + l times q_odd / 16, its low code l times the rest of
            // q_even; the sum is that of the coefficients as rounded
            const int k = j & 2;
            float lo = q[8 * i + k + 1] * 0.0625f, hi = q[8 * i + 4 + k + 1] * 0.0625f;
            if (!(j & 1)) {
              lo = q[8 * i + k] - lo;
              hi = q[8 * i + 4 + k] - hi;
            }
            qf[i][j] = half2_bits(lo * up, hi * up);
            const float2 r = half2_floats(qf[i][j]);
            sum += (r.x + r.y) * (j & 1 ? 17.0f : 1.0f);
          }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        const float f = P.softmax_scale * (1.4426950408889634f * 0.08838834764831845f) * pow2f(-sh);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float fj = __shfl_sync(0xffffffffu, f, (2 * t + j) * 4);
          fa[j] = fj * 0x1p24f;
          fz[j] = fj * __shfl_sync(0xffffffffu, sum, (2 * t + j) * 4);
          m[j] = -INFINITY;
          ref[j] = 0.0f;
          l[j] = zs[j] = zs[2 + j] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
        ev = -14;
        fresh = true;
      }
      const int todo = min(w.tiles - w.tile, w.left);
      for (int it = 0; it < todo; ++it) {
        // the tile's copies have landed and its scales are stored, and every warp
        // is done with the stage that is filled next
        wait_copies<S::kStages - 2>();
        store_scales();
        __syncthreads();
        fetch();
        const int s = stage;
        if (++stage == S::kStages) stage = 0;
        const uint8_t* kb = smem + s * S::kStage + tok0 * S::kRow + hw * 64;
        const uint8_t* vb = kb + S::kCodes;
        const uint8_t* scales = smem + s * S::kStage + 2 * S::kCodes;
        const uint16_t* sb = reinterpret_cast<const uint16_t*>(scales) + tok0 * HB + hw;
        const uint32_t hidden =
            __ballot_sync(0xffffffffu, scales[S::kScales + tok0 + lane % S::kTok]);
        float sc[MB][2][2];                // [block][row g or g + 8][column], minus ref
        float vs[MB][2];                   // value scale of the row, times 2^(15 - kSlack - ev)
        const float vup = pow2f(15 - kSlack - ev);
        float vtop = 0.0f;
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          const uint4 ka = *reinterpret_cast<const uint4*>(kb + (mb * 16 + mine) * S::kRow + t * 16);
          const uint4 kc =
              *reinterpret_cast<const uint4*>(kb + (mb * 16 + 8 + mine) * S::kRow + t * 16);
          const uint32_t xa[4] = {ka.x, ka.y, ka.z, ka.w}, xc[4] = {kc.x, kc.y, kc.z, kc.w};
          float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            mma16816(c, xa[i] & 0x000f000fu, xc[i] & 0x000f000fu, xa[i] & 0x00ff00ffu,
                     xc[i] & 0x00ff00ffu, qf[i][0], qf[i][1]);
            const uint32_t ya = __byte_perm(xa[i], 0, 0x4341), yc = __byte_perm(xc[i], 0, 0x4341);
            mma16816(c, ya & 0x000f000fu, yc & 0x000f000fu, ya, yc, qf[i][2], qf[i][3]);
          }
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const uint16_t* at = sb + (mb * 16 + 8 * r + mine) * HB;
            const float ks = f16_bits_to_f32(at[0]);
            const float kz = f16_bits_to_f32(at[S::kArray / 2]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              sc[mb][r][j] = fmaf(ks, fmaf(fa[j], c[2 * r + j], -kz * fz[j]), -ref[j]);
            vs[mb][r] = f16_bits_to_f32(at[S::kArray]) * vup;
          }
          vtop = fmax3(vtop, fabsf(vs[mb][0]), fabsf(vs[mb][1]));
        }
        if (hidden != 0) {
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int r = 0; r < 2; ++r)
              if (hidden >> (mb * 16 + 8 * r + mine) & 1)
                sc[mb][r][0] = sc[mb][r][1] = -INFINITY;
        }
        // ---- running maximum, and the value scales' power of two.  Both stay as
        // they are until a score passes the maximum by kSlack or a value scale its
        // power of two, which is seldom behind the first tile.
        float stop[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int j = 0; j < 2; ++j) stop[j] = fmax3(stop[j], sc[mb][0][j], sc[mb][1][j]);
        if (fresh || __any_sync(0xffffffffu, fmaxf(stop[0], stop[1]) > (float)kSlack ||
                                                 vtop > (float)(1 << (15 - kSlack)))) {
          fresh = hidden == 0xffffffffu;
          float keep[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float mt = fmaxf(m[j], max_over_rows(stop[j]) + ref[j]);
            const float next = mt == -INFINITY ? 0.0f : mt;
            keep[j] = exp2_(m[j] - next);
            l[j] *= keep[j];
#pragma unroll
            for (int mb = 0; mb < MB; ++mb)
#pragma unroll
              for (int r = 0; r < 2; ++r) sc[mb][r][j] += ref[j] - next;
            m[j] = mt;
            ref[j] = next;
          }
          // every value scale seen is below 2^ev
          const uint32_t bits = redux_max(__float_as_uint(vtop));
          const int up = max((int)(bits >> 23) - 126 - (15 - kSlack), 0);
          const float down = pow2f(-up);
          ev += up;
#pragma unroll
          for (int mb = 0; mb < MB; ++mb)
#pragma unroll
            for (int r = 0; r < 2; ++r) vs[mb][r] *= down;
          keep[0] *= down;
          keep[1] *= down;
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) o[i][j] *= keep[j & 1];
#pragma unroll
          for (int j = 0; j < 4; ++j) zs[j] *= keep[j & 1];
        }
        // p s' 2^(15 - kSlack - ev) < 2^15: 11 bits for weights down to 2^-23 of the
        // maximum at the largest value scale, none lost above 2^-33
        uint32_t pf[MB][2];
#pragma unroll
        for (int mb = 0; mb < MB; ++mb)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float p0 = exp2_(sc[mb][r][0]), p1 = exp2_(sc[mb][r][1]);
            l[0] += p0;
            l[1] += p1;
            pf[mb][r] = transpose8x8(half2_bits(p0 * vs[mb][r], p1 * vs[mb][r]));
          }
        // ---- values
#pragma unroll
        for (int mb = 0; mb < MB; ++mb) {
          // the zero points as one more dimension (every row the same)
          const uint16_t* zv = sb + 3 * (S::kArray / 2) + mb * 16 * HB;
          const uint32_t z01 = zv[even * HB] | (uint32_t)zv[odd * HB] << 16;
          const uint32_t z23 = zv[(8 + even) * HB] | (uint32_t)zv[(8 + odd) * HB] << 16;
          mma16816(zs, z01, z01, z23, z23, pf[mb][0], pf[mb][1]);
          uint2 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = *reinterpret_cast<const uint2*>(
                vb + (mb * 16 + 8 * (i >> 1) + (i & 1 ? odd : even)) * S::kRow + g * 8);
#pragma unroll
          for (int j = 0; j < 4; ++j) {     // 4 dimensions of the lane's 16
            const uint32_t sel = j & 1 ? 0x7632u : 0x5410u;
            const uint32_t y01 = j < 2 ? __byte_perm(x[0].x, x[1].x, sel)
                                       : __byte_perm(x[0].y, x[1].y, sel);
            const uint32_t y23 = j < 2 ? __byte_perm(x[2].x, x[3].x, sel)
                                       : __byte_perm(x[2].y, x[3].y, sel);
            mma16816(o[2 * j], y01 & 0x000f000fu, y01 & 0x00ff00ffu, y23 & 0x000f000fu,
                     y23 & 0x00ff00ffu, pf[mb][0], pf[mb][1]);
            const uint32_t h01 = __byte_perm(y01, 0, 0x4341), h23 = __byte_perm(y23, 0, 0x4341);
            mma16816(o[2 * j + 1], h01 & 0x000f000fu, h01, h23 & 0x000f000fu, h23, pf[mb][0],
                     pf[mb][1]);
          }
        }
      }
      // ---- end of the unit in this CTA: values in real units
      float r[2][16];
      {
        const float down = pow2f(ev - (15 - kSlack));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          l[j] = sum_over_rows(l[j]);
          const float z = zs[j];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            r[j][2 * i] = (o[i][j] * 0x1p24f - z) * down;
            r[j][2 * i + 1] = ((o[i][2 + j] - o[i][j]) * 0x1p20f - z) * down;
          }
        }
      }
      if constexpr (S::kSplit > 1) {
        // join the head's warps, two by two
#pragma unroll
        for (int half = S::kSplit / 2; half > 0; half >>= 1) {
          float* slot = join + (hw * (S::kSplit / 2) + part % half) * kPartFloats;
          if (part >= half && part < 2 * half) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              float4* to = reinterpret_cast<float4*>(slot + (2 * t + j) * 128 + 16 * g);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                to[i] = make_float4(r[j][4 * i], r[j][4 * i + 1], r[j][4 * i + 2], r[j][4 * i + 3]);
              slot[kCols * 128 + 2 * t + j] = m[j];
              slot[kCols * 128 + kCols + 2 * t + j] = l[j];
            }
          }
          __syncthreads();
          if (part < half) {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float m2 = slot[kCols * 128 + 2 * t + j];
              const float mt = fmaxf(m[j], m2), rf = mt == -INFINITY ? 0.0f : mt;
              const float a = exp2_(m[j] - rf), b = exp2_(m2 - rf);
              const float4* from = reinterpret_cast<const float4*>(slot + (2 * t + j) * 128 + 16 * g);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float4 v = from[i];
                r[j][4 * i] = r[j][4 * i] * a + v.x * b;
                r[j][4 * i + 1] = r[j][4 * i + 1] * a + v.y * b;
                r[j][4 * i + 2] = r[j][4 * i + 2] * a + v.z * b;
                r[j][4 * i + 3] = r[j][4 * i + 3] * a + v.w * b;
              }
              l[j] = l[j] * a + slot[kCols * 128 + kCols + 2 * t + j] * b;
              m[j] = mt;
            }
          }
          __syncthreads();
        }
      }
      const bool whole = todo == w.tiles;
      if (!ALONE && threadIdx.x == 0) {      // for the join
        Span* span = span_of(P, w.b, blocks, w.hb, chunks, w.chunk);
        if (w.tile == 0) span->first = 2 * (int)blockIdx.x + (segment ? 1 : 0);
        if (w.tile + todo == w.tiles) span->last = (int)blockIdx.x;
      }
      if (part == 0) {
        if (whole) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float inv = l[j] > 0.0f ? 1.0f / l[j] : 0.0f;
#pragma unroll
            for (int i = 0; i < 16; ++i) r[j][i] *= inv;
            store_result(P, r[j], w.b, kh * group + col0 + 2 * t + j, kh, 2 * t + j < columns);
          }
        } else {
          float* slot = static_cast<float*>(P.workspace) +
                        (((int64_t)blockIdx.x * 2 + (segment ? 1 : 0)) * kWarps + hw) * kPartFloats;
#pragma unroll
          for (int j = 0; j < 2; ++j)
            if (2 * t + j < columns) {
              float4* to = reinterpret_cast<float4*>(slot + (2 * t + j) * 128 + 16 * g);
#pragma unroll
              for (int i = 0; i < 4; ++i)
                to[i] = make_float4(r[j][4 * i], r[j][4 * i + 1], r[j][4 * i + 2], r[j][4 * i + 3]);
              if (g == 0)
                reinterpret_cast<float2*>(slot + kCols * 128)[2 * t + j] = make_float2(m[j], l[j]);
            }
        }
      }
      ++segment;
      w.tile += todo - 1;
      w.left -= todo - 1;
      step<TILE>(P, most, blocks, chunks, w);
    }
  }
}

// ---- joining the partial sums of the units that more than one CTA worked on, in
// CTA order.
constexpr int kRowWarps = 4;                  // warps with a row each, when there are many rows

// Where the partial sums of a unit lie: `n` of them (one that is whole in its CTA has
// none), from that CTA on.
struct Parts {
  const float* base;
  int n, second;
  __device__ __forceinline__ const float* slot(int i) const {
    return base + (i * 2 + (i == 0 ? second : 0)) * kWarps * kPartFloats;
  }
};
template <int HB>
__device__ __forceinline__ Parts parts_of(const AttnArgs& P, int64_t b, int kh, int chunk) {
  const int chunks = (P.q_heads / P.kv_heads + kCols - 1) / kCols;
  const Span span = *span_of(P, b, P.kv_heads / HB, kh / HB, chunks, chunk);
  // a sequence without a visible token has no tile and no span
  const bool any = sequence(P, longest(P), b).vis > 0;
  const int c0 = span.first >> 1;
  return Parts{static_cast<const float*>(P.workspace) +
                   ((int64_t)c0 * 2 * kWarps + kh % HB) * kPartFloats,
               any ? span.last - c0 + 1 : 0, span.first & 1};
}

// Maximum, sum and values (4 dimensions a lane) of column `col` over the partial
// sums i0, i0 + by, ...; AHEAD of them are loaded at a time, with a running maximum.
// (A CTA a row: 10, 131071 tokens 42.0 us and 42.7 with 4; a warp a row: 6, 64 windows of
// 1028 tokens 27.4 us and 27.8 with 8 or 10; both when finding the CTAs overlapped the wait.)
struct Joined {
  float m, l;
  float4 v;
};
template <int AHEAD>
__device__ __forceinline__ Joined sum_parts(const Parts& p, int col, int i0, int by) {
  const int lane = threadIdx.x & 31;
  Joined r{-INFINITY, 0.0f, make_float4(0.0f, 0.0f, 0.0f, 0.0f)};
  for (; i0 < p.n; i0 += AHEAD * by) {
    float pm[AHEAD], pl[AHEAD];
    float4 v[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + k * by;
      pm[k] = -INFINITY;
      pl[k] = 0.0f;
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i < p.n) {
        const float* s = p.slot(i);
        const float2 ml = reinterpret_cast<const float2*>(s + kCols * 128)[col];
        pm[k] = ml.x;
        pl[k] = ml.y;
        v[k] = *reinterpret_cast<const float4*>(s + col * 128 + 4 * lane);
      }
    }
    float top = r.m;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) top = fmaxf(top, pm[k]);
    const float ref = top == -INFINITY ? 0.0f : top, keep = exp2_(r.m - ref);
    r.m = top;
    r.l *= keep;
    r.v.x *= keep;
    r.v.y *= keep;
    r.v.z *= keep;
    r.v.w *= keep;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const float f = exp2_(pm[k] - ref);
      r.l = fmaf(f, pl[k], r.l);
      r.v.x = fmaf(f, v[k].x, r.v.x);
      r.v.y = fmaf(f, v[k].y, r.v.y);
      r.v.z = fmaf(f, v[k].z, r.v.z);
      r.v.w = fmaf(f, v[k].w, r.v.w);
    }
  }
  return r;
}
// Signs of a lane's 4 dimensions of a cached head.
__device__ __forceinline__ uint32_t join_signs(const AttnArgs& P, int kh) {
  const int at = kh * 128 + 4 * (threadIdx.x & 31);
  return P.v_signs ? *reinterpret_cast<const uint32_t*>(P.v_signs + at) : 0;
}
// A warp rotates a joined row back, 4 dimensions a lane, and stores it.
__device__ __forceinline__ void store_joined(const AttnArgs& P, float l, float4 v, uint32_t signs,
                                             int64_t b, int qh) {
  const int lane = threadIdx.x & 31;
  const float inv = l == 0.0f ? 0.0f : 0.08838834764831845f / l;
  float r[4] = {v.x + v.y, v.x - v.y, v.z + v.w, v.z - v.w};
  const float a0 = r[0], a1 = r[1];
  r[0] = (a0 + r[2]) * inv;
  r[1] = (a1 + r[3]) * inv;
  r[2] = (a0 - r[2]) * inv;
  r[3] = (a1 - r[3]) * inv;
#pragma unroll
  for (int st = 1; st < 32; st <<= 1) {
    const float own = (lane & st) ? -1.0f : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = fmaf(own, r[i], __shfl_xor_sync(0xffffffffu, r[i], st));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    r[i] = __uint_as_float(__float_as_uint(r[i]) ^ (signs << (24 - 8 * i) & 0x80000000u));
  const __nv_bfloat162 lo = __floats2bfloat162_rn(r[0], r[1]), hi = __floats2bfloat162_rn(r[2], r[3]);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(P.out) + (b * P.q_heads + qh) * 128 + 4 * lane) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
}

// Many rows: a CTA takes (sequence, cached head, chunk of its query heads), a warp
// a query head at a time.
template <int HB>
__global__ void __launch_bounds__(32 * kRowWarps) k_join_rows(AttnArgs P) {
  const int warp = threadIdx.x >> 5;
  const int group = P.q_heads / P.kv_heads, chunks = (group + kCols - 1) / kCols;
  const int64_t b = blockIdx.x;
  const int kh = blockIdx.y / chunks, chunk = blockIdx.y - kh * chunks;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Parts p = parts_of<HB>(P, b, kh, chunk);
  const uint32_t signs = join_signs(P, kh);
  if (p.n < 2) return;
  const int columns = min(kCols, group - chunk * kCols);
  for (int col = warp; col < columns; col += kRowWarps) {
    const Joined r = sum_parts<6>(p, col, 0, 1);
    store_joined(P, r.l, r.v, signs, b, kh * group + chunk * kCols + col);
  }
}

// Fewer rows, which may have partial sums of many CTAs: a CTA takes one.
template <int HB, int kJoinWarps>
__global__ void __launch_bounds__(32 * kJoinWarps) k_join_wide(AttnArgs P) {
  __shared__ float2 ml[kJoinWarps];
  __shared__ __align__(16) float red[kJoinWarps][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t b = blockIdx.x;
  const int qh = blockIdx.y, group = P.q_heads / P.kv_heads, kh = qh / group;
  const int chunk = (qh - kh * group) / kCols, col = (qh - kh * group) % kCols;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Parts p = parts_of<HB>(P, b, kh, chunk);
  const uint32_t signs = warp == 0 ? join_signs(P, kh) : 0;
  if (p.n < 2) return;
  const Joined r = sum_parts<10>(p, col, warp, kJoinWarps);
  *reinterpret_cast<float4*>(&red[warp][4 * lane]) = r.v;
  if (lane == 0) ml[warp] = make_float2(r.m, r.l);
  __syncthreads();
  if (warp > 0) return;
  float top = -INFINITY, ls = 0.0f;
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) top = fmaxf(top, ml[k].x);
  const float ref = top == -INFINITY ? 0.0f : top;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int k = 0; k < kJoinWarps; ++k) {
    const float f = exp2_(ml[k].x - ref);
    const float4 o = *reinterpret_cast<const float4*>(&red[k][4 * lane]);
    ls = fmaf(f, ml[k].y, ls);
    v.x = fmaf(f, o.x, v.x);
    v.y = fmaf(f, o.y, v.y);
    v.z = fmaf(f, o.z, v.z);
    v.w = fmaf(f, o.w, v.w);
  }
  store_joined(P, ls, v, signs, b, qh);
}

PageDiv page_div(int page_size) {
  PageDiv d{0, 0};
  if (page_size > 1) {
    uint32_t l = 1;
    while ((1u << l) < (uint32_t)page_size) ++l;
    d.mul = (uint32_t)(((uint64_t(1) << (31 + l)) + page_size - 1) / page_size);
    d.shift = l - 1;
  }
  return d;
}

cudaError_t multiprocessors(int* out) {
  // looked up once a device
  constexpr int kDevices = 64;
  static std::atomic<int> known[kDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= kDevices || (*out = known[dev].load(std::memory_order_relaxed)) == 0) {
    e = cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev < kDevices) known[dev].store(*out, std::memory_order_relaxed);
  }
  return cudaSuccess;
}

cudaError_t launch_alone(const AttnArgs& P, int units, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute((const void*)k_attn<1, true>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)Shape<1>::kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  const cudaLaunchConfig_t cfg =
      dependent_launch(dim3((unsigned)units), kThreads, Shape<1>::kSmem, s, attr);
  return cudaLaunchKernelEx(&cfg, k_attn<1, true>, P, page_div(P.page_size));
}

template <int HB>
cudaError_t launch(const AttnArgs& P, int sms, cudaStream_t s) {
  // (a context's, so set at every call)
  cudaError_t e = cudaFuncSetAttribute((const void*)k_attn<HB, false>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)Shape<HB>::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = 2 * sms < kMaxCtas ? 2 * sms : kMaxCtas;
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg =
      dependent_launch(dim3((unsigned)grid), kThreads, Shape<HB>::kSmem, s, attr);
  e = cudaLaunchKernelEx(&cfg, k_attn<HB, false>, P, page_div(P.page_size));
  if (e != cudaSuccess) return e;
  // A row's CTA of 16 warps, 4 or 1, as far as they all run at a time: 32
  // sequences of 32 heads (1024 rows) took 24.4 us with 4 warps and 25.5 with 1,
  // 2048 rows 31.0 with 4 and 28.1 with 1 (before the join held 4 dimensions a lane).
  const int64_t rows = P.batch * P.q_heads;
  if (rows <= 8 * sms) {
    const dim3 each((unsigned)P.batch, (unsigned)P.q_heads);
    const bool few = rows <= 2 * sms;
    cfg = dependent_launch(each, few ? 32 * 16 : 32 * 4, 0, s, attr);
    return few ? cudaLaunchKernelEx(&cfg, k_join_wide<HB, 16>, P)
               : cudaLaunchKernelEx(&cfg, k_join_wide<HB, 4>, P);
  }
  const int chunks = (P.q_heads / P.kv_heads + kCols - 1) / kCols;
  cfg = dependent_launch(dim3((unsigned)P.batch, (unsigned)(P.kv_heads * chunks)),
                         32 * kRowWarps, 0, s, attr);
  return cudaLaunchKernelEx(&cfg, k_join_rows<HB>, P);
}

}  // namespace at

size_t attn_workspace_bytes(int64_t batch, int q_heads, int kv_heads) {
  // as many units as there are with one cached head each
  const int64_t units = batch * kv_heads * ((q_heads / kv_heads + at::kCols - 1) / at::kCols);
  return at::kPartBytes + sizeof(at::Span) * (size_t)(units + (units & 1));
}

cudaError_t launch_attn_decode(const AttnArgs& args, cudaStream_t s) {
  AttnArgs P = args;
  if (P.num_slots == 0) P.table_width = 0;    // no row to read: every sequence is empty
  int sms = 0;
  const cudaError_t e = at::multiprocessors(&sms);
  if (e != cudaSuccess) return e;
  const int chunks = (P.q_heads / P.kv_heads + at::kCols - 1) / at::kCols;
  const int64_t units = P.batch * P.kv_heads * chunks, keep = (int64_t)P.window + P.sinks;
  const int64_t longest = P.table_width * P.page_size;
  if (units <= 2 * sms && (P.window > 0 && keep < longest ? keep : longest) <= at::kAloneTokens)
    return at::launch_alone(P, (int)units, s);
  // The widest block of heads whose rows and scales stay whole.  (8 cached heads in blocks
  // of 8, 4, 2, 1: 32 sequences of 300 to 4096 tokens 23.5, 24.8, 28.8, 33.8 us; 131071
  // tokens 42.8, 43.0, 50.2, 55.5; 64 behind a window 27.7, 30.3, 37.7, 44.9.  Blocks of 2
  // spill 32 bytes, the others nothing.)
  if (P.kv_heads % 8 == 0) return at::launch<8>(P, sms, s);
  if (P.kv_heads % 4 == 0) return at::launch<4>(P, sms, s);
  if (P.kv_heads % 2 == 0) return at::launch<2>(P, sms, s);
  return at::launch<1>(P, sms, s);
}

}  // namespace kq
