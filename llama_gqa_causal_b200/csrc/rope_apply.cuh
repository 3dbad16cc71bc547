// Rotation of q and k by a cos/sin table, and tables whose frequencies are
// scaled for long contexts.
//
// rope_table_scaled_kernel: cos, sin (pos * w'_i), times a gain, from host-made
// frequencies w'_i.  rope_apply_*_kernel: every head of every token turned by
// its token's row, pair i of the first R dimensions (a, z) -> (a c - z s,
// z c + a s); the transposed map (the gradient) has -s in place of s.  fp32
// arithmetic, one rounding.
#pragma once
#include "common.cuh"

namespace la {
namespace ra {
constexpr int kMaxHalf = 256;  // frequencies of a scaled table: head_dim <= 512
constexpr int THREADS = 256;
}  // namespace ra

struct ScaledFreqs {
  double inv[ra::kMaxHalf];
};

__global__ void __launch_bounds__(ra::THREADS)
    rope_table_scaled_kernel(const long long* __restrict__ pos, long long n_rows, int half,
                             double gain, float* __restrict__ cos_out, float* __restrict__ sin_out,
                             const __grid_constant__ ScaledFreqs freqs) {
  const long long total = n_rows * half;
  for (long long idx = blockIdx.x * (long long)blockDim.x + threadIdx.x; idx < total;
       idx += (long long)gridDim.x * blockDim.x) {
    const long long r = idx / half;
    const int i = static_cast<int>(idx - r * half);
    double s, c;
    sincos(static_cast<double>(pos[r]) * freqs.inv[i], &s, &c);
    const float cf = static_cast<float>(c * gain), sf = static_cast<float>(s * gain);
    const long long o = r * 2 * half + i;
    cos_out[o] = cf;
    cos_out[o + half] = cf;
    sin_out[o] = sf;
    sin_out[o + half] = sf;
  }
}

// One of the two tensors of a rotation: strides in elements of batch entry,
// token and head; the dimensions of a head are adjacent.
struct RopeSide {
  const void* x;
  void* y;
  long long xb, xs, xh, yb, ys, yh;
  int heads;
};
struct RopeApplyParams {
  RopeSide side[2];  // q, k (k: no heads if absent)
  const float* cos;  // [tokens, R]
  const float* sin;
  long long tokens;  // bsz * seq
  int seq, D, R;
  float sign;        // 1, or -1 for the transposed map
};

__device__ __forceinline__ float ra_load(const float* p) { return *p; }
__device__ __forceinline__ float ra_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void ra_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void ra_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Any even R, any alignment: a thread per pair or per copied element.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(ra::THREADS) rope_apply_any_kernel(RopeApplyParams p) {
  const int half = p.R / 2;
  const int per_head = half + (p.D - p.R);
  const long long heads = p.side[0].heads + p.side[1].heads;
  const long long total = p.tokens * heads * per_head;
  for (long long idx = blockIdx.x * (long long)blockDim.x + threadIdx.x; idx < total;
       idx += (long long)gridDim.x * blockDim.x) {
    const long long row = idx / per_head;
    const int e = static_cast<int>(idx - row * per_head);
    const long long tok = row / heads;
    int h = static_cast<int>(row - tok * heads);
    const bool is_k = h >= p.side[0].heads;
    const RopeSide& sd = is_k ? p.side[1] : p.side[0];
    if (is_k) h -= p.side[0].heads;
    const long long b = tok / p.seq, s = tok - b * p.seq;
    const T* x = static_cast<const T*>(sd.x) + b * sd.xb + s * sd.xs + h * sd.xh;
    T* y = static_cast<T*>(sd.y) + b * sd.yb + s * sd.ys + h * sd.yh;
    if (e < half) {
      const float c = p.cos[tok * p.R + e], sn = p.sign * p.sin[tok * p.R + e];
      const int d0 = INTERLEAVED ? 2 * e : e, d1 = INTERLEAVED ? 2 * e + 1 : e + half;
      const float a = ra_load(x + d0), z = ra_load(x + d1);
      ra_store(y + d0, fmaf(a, c, -z * sn));
      ra_store(y + d1, fmaf(z, c, a * sn));
    } else {
      y[p.R + e - half] = x[p.R + e - half];
    }
  }
}

}  // namespace la
