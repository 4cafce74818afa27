// Attention of one new token per sequence over the paged INT4 KV cache that
// kq_rht_quant_int4_kv writes (QuaRot reviews, final comments: the KV cache at
// 4 bits with a per-head 128-point Hadamard).  Keys and values are stored
// rotated, so the query is rotated on the way in (q . k is unchanged when both
// carry the rotation) and the result rotated back on the way out.
//
// One CTA per (sequence, query head), a thread per token for the scores and a
// thread per dimension for the values, with a running maximum and sum.
#include <cuda_bf16.h>

#include <cstdint>

#include "kq_internal.h"

namespace kq {
namespace at {

__global__ void __launch_bounds__(128) k_attn(AttnArgs P) {
  __shared__ float qs[128], ps[128];
  __shared__ double red[40];
  __shared__ int64_t slots[128];
  const int d = threadIdx.x;
  const int64_t b = blockIdx.x;
  const int h = blockIdx.y, kh = h / (P.q_heads / P.kv_heads);
  auto rotate = [&] {                 // unnormalized H_128 of qs
    for (int st = 1; st < 128; st <<= 1) {
      __syncthreads();
      const float a = qs[d], c = qs[d ^ st];
      __syncthreads();
      qs[d] = (d & st) ? c - a : a + c;
    }
    __syncthreads();
  };
  const int64_t qi = (b * P.q_heads + h) * 128 + d;
  float q = __bfloat162float(static_cast<const __nv_bfloat16*>(P.q)[qi]);
  if (P.k_signs && P.k_signs[kh * 128 + d] < 0) q = -q;
  qs[d] = q * 0.08838834764831845f;
  rotate();
  int64_t len = P.seq_lens[b];
  const int64_t most = P.table_width * P.page_size;
  len = len < 0 ? 0 : len > most ? most : len;
  const int64_t keep = (int64_t)P.window + P.sinks;
  const int64_t skip = P.window > 0 && len > keep ? len - keep : 0;
  const int64_t vis = len - skip;
  const int row = P.kv_heads;
  float m = -INFINITY, l = 0.0f, o = 0.0f;
  for (int64_t t0 = 0; t0 < vis; t0 += 128) {
    __syncthreads();
    int64_t slot = -1;
    const int64_t v = t0 + d;
    if (v < vis) {
      const int64_t pos = v < P.sinks ? v : v + skip;
      const int64_t page = P.block_table[b * P.table_width + pos / P.page_size];
      slot = page * P.page_size + pos % P.page_size;
      if (page < 0 || slot >= P.num_slots) slot = -1;
    }
    float sc = -INFINITY;
    if (slot >= 0) {
      const uint8_t* c = P.k_codes + (slot * row + kh) * 64;
      const float s = f16_bits_to_f32(P.k_scales[slot * row + kh]);
      const float z = f16_bits_to_f32(P.k_zeros[slot * row + kh]);
      float a = 0.0f;
      for (int i = 0; i < 64; ++i) {
        const uint32_t w = c[i];
        a = fmaf(qs[2 * i], (float)(w & 15u) - z, a);
        a = fmaf(qs[2 * i + 1], (float)(w >> 4) - z, a);
      }
      sc = a * s * P.softmax_scale;
    }
    slots[d] = slot;
    const float mt = fmaxf(m, block_max(sc, red));
    const float ref = mt == -INFINITY ? 0.0f : mt;
    const float keep_f = expf(m - ref);
    const float p = expf(sc - ref);
    ps[d] = p;
    l = l * keep_f + (float)block_sum_d((double)p, red);
    o *= keep_f;
    m = mt;
    __syncthreads();
    const int n = vis - t0 < 128 ? (int)(vis - t0) : 128;
    for (int t = 0; t < n; ++t) {
      const int64_t sl = slots[t];
      if (sl < 0) continue;
      const uint32_t w = P.v_codes[(sl * row + kh) * 64 + d / 2];
      const float u = (float)((d & 1) ? w >> 4 : w & 15u);
      o = fmaf(ps[t], (u - f16_bits_to_f32(P.v_zeros[sl * row + kh])) *
                          f16_bits_to_f32(P.v_scales[sl * row + kh]), o);
    }
  }
  __syncthreads();
  qs[d] = l > 0.0f ? o / l * 0.08838834764831845f : 0.0f;
  rotate();
  float r = qs[d];
  if (P.v_signs && P.v_signs[kh * 128 + d] < 0) r = -r;
  static_cast<__nv_bfloat16*>(P.out)[qi] = __float2bfloat16_rn(r);
}

}  // namespace at

size_t attn_workspace_bytes(int64_t batch, int q_heads, int kv_heads) {
  (void)batch; (void)q_heads; (void)kv_heads;
  return 16;
}

cudaError_t launch_attn_decode(const AttnArgs& P, cudaStream_t s) {
  at::k_attn<<<dim3((unsigned)P.batch, (unsigned)P.q_heads), 128, 0, s>>>(P);
  return cudaGetLastError();
}

}  // namespace kq
