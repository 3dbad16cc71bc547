// Decode for a batch whose sequences share a prefix: one query row per head
// against the prefix's rows and the sequence's own, in one softmax.
//
// One block per (head, batch entry); its four warps take every fourth key, a
// lane D / 32 dimensions, and merge their running (max, sum, output).
#pragma once
#include "decode_bf16.cuh"

namespace la {

struct DecodePrefixParams {
  const __nv_bfloat16* q;      // [b, H, D]
  const __nv_bfloat16* k_pre;  // prefix rows, strides below
  const __nv_bfloat16* v_pre;
  long long kp_head, kp_row, vp_head, vp_row;  // in elements
  const __nv_bfloat16* k_new;  // [b, Hkv, D] or null
  const __nv_bfloat16* v_new;
  __nv_bfloat16* k_cache;      // [b, Hkv, L, D]
  __nv_bfloat16* v_cache;
  const int* lens;
  __nv_bfloat16* out;          // [b, H * D]
  int prefix_len, H, Hkv, L, group;
  float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(128) decode_prefix_plain_kernel(DecodePrefixParams p) {
  constexpr int VEC = D / 32;
  __shared__ float so[4][D], sm[4], sl[4];
  const int h = blockIdx.x, b = blockIdx.y, kvh = h / p.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int append = p.k_new != nullptr;
  const int len = attend_len(p.lens[b], p.L, append);
  const int row_new = append ? len - 1 : -1;
  const size_t bh = static_cast<size_t>(b) * p.Hkv + kvh;
  float q[VEC], o[VEC], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    q[v] = __bfloat162float(p.q[(static_cast<size_t>(b) * p.H + h) * D + lane * VEC + v]);
    o[v] = 0.f;
  }
  auto key = [&](const __nv_bfloat16* kr, const __nv_bfloat16* vr) {
    float x = 0.f;
#pragma unroll
    for (int v = 0; v < VEC; ++v) x = fmaf(q[v], __bfloat162float(kr[lane * VEC + v]), x);
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) x += __shfl_xor_sync(0xffffffffu, x, s);
    x *= p.scale_log2;
    const float m_new = fmaxf(m, x);
    const float alpha = m == -INFINITY ? 0.f : exp2f(m - m_new);
    const float w = exp2f(x - (m_new == -INFINITY ? 0.f : m_new));  // (a NaN score stays one)
    l = fmaf(l, alpha, w);
#pragma unroll
    for (int v = 0; v < VEC; ++v) o[v] = fmaf(o[v], alpha, w * __bfloat162float(vr[lane * VEC + v]));
    m = m_new;
  };
  for (int j = warp; j < p.prefix_len; j += 4)
    key(p.k_pre + kvh * p.kp_head + j * p.kp_row, p.v_pre + kvh * p.vp_head + j * p.vp_row);
  for (int j = warp; j < len; j += 4) {
    if (j == row_new) key(p.k_new + bh * D, p.v_new + bh * D);
    else key(p.k_cache + (bh * p.L + j) * D, p.v_cache + (bh * p.L + j) * D);
  }
  if (append && h % p.group == 0 && warp == 0) {
    for (int d = lane; d < D; d += 32) {
      p.k_cache[(bh * p.L + row_new) * D + d] = p.k_new[bh * D + d];
      p.v_cache[(bh * p.L + row_new) * D + d] = p.v_new[bh * D + d];
    }
  }
  if (lane == 0) {
    sm[warp] = m;
    sl[warp] = l;
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) so[warp][lane * VEC + v] = o[v];
  __syncthreads();
  float top = -INFINITY, sum = 0.f;
  for (int w = 0; w < 4; ++w) top = fmaxf(top, sm[w]);
  if (threadIdx.x < D) {
    float acc = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float f = sm[w] == -INFINITY ? 0.f : exp2f(sm[w] - top);
      sum = fmaf(f, sl[w], sum);
      acc = fmaf(f, so[w][threadIdx.x], acc);
    }
    p.out[(static_cast<size_t>(b) * p.H + h) * D + threadIdx.x] =
        __float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum);
  }
}

}  // namespace la
