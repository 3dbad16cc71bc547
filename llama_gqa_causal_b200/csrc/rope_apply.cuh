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
constexpr int HB = 4;          // heads of a thread of the vector rotation
}  // namespace ra

struct ScaledFreqs {
  double inv[ra::kMaxHalf];
};

// sin and cos of x, |x| < 2^40, to one step of fp32 with the gain's rounding, where
// the fp64 functions, rounded once, would be off by half a step: 131072 rows of 128
// take 26.7 us against 68.  x is reduced in
// fp64 by the nearest multiple k of pi/2, held as a sum of two doubles, to r in
// [-pi/4, pi/4]; r = rf + rl (rf the nearest float); the Taylor polynomials of
// sin and cos to r^9 and r^10 (the next terms are below 2^-28 there) are taken
// of rf in fp32, and rl enters through the derivative; k mod 4 turns the pair.
// Six fp64 operations instead of the library's two fp64 polynomials.
__device__ __forceinline__ void sincos_reduced(double x, float& s, float& c) {
  constexpr double kRound = 6755399441055744.0;  // 1.5 * 2^52: x + kRound holds rint(x) in its low bits
  const double t = fma(x, 0.63661977236758134308, kRound);  // 2 / pi
  const double k = t - kRound;
  const int quadrant = __double2loint(t) & 3;
  double r = fma(-k, 1.57079632679489655800, x);   // pi / 2, its first double
  r = fma(-k, 6.12323399573676603587e-17, r);      // and what is left of it
  const float rf = static_cast<float>(r), rl = static_cast<float>(r - static_cast<double>(rf));
  const float r2 = rf * rf;
  float ps = fmaf(r2, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, -1/7!
  ps = fmaf(ps, r2, 8.3333333e-3f);                    // 1/5!
  ps = fmaf(ps, r2, -0.16666667f);
  float pc = fmaf(r2, -2.7557319e-7f, 2.4801587e-5f);  // -1/10!, 1/8!
  pc = fmaf(pc, r2, -1.3888889e-3f);                   // -1/6!
  pc = fmaf(pc, r2, 4.1666667e-2f);                    // 1/4!
  pc = fmaf(pc, r2, -0.5f);
  const float sn = rf + fmaf(ps * r2, rf, rl);    // cos(rf) rl = rl to within 2^-26
  const float cs = 1.f + fmaf(pc, r2, -rf * rl);
  s = (quadrant & 1) ? cs : sn;
  c = (quadrant & 1) ? sn : cs;
  s = (quadrant & 2) ? -s : s;
  c = ((quadrant + 1) & 2) ? -c : c;
}

// Threads of a block: rows x (half / VEC), each with VEC adjacent frequencies
// that it keeps in registers while it walks the rows (the frequencies lie in
// the parameter bank, where lanes with different indexes are served one by
// one).  Bound by its writes, 8 bytes for each of head_dim entries of a row:
// 131072 rows of 128 with the library's fp64 sincos took 68 us.
template <int VEC>
__global__ void __launch_bounds__(ra::THREADS)
    rope_table_scaled_kernel(const long long* __restrict__ pos, long long n_rows, int half,
                             double gain, bool stream_out, float* __restrict__ cos_out,
                             float* __restrict__ sin_out,
                             const __grid_constant__ ScaledFreqs freqs) {
  const int per_row = half / VEC;
  const int rows_per_block = blockDim.x / per_row;
  const int i = static_cast<int>(threadIdx.x % per_row) * VEC;
  double inv[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) inv[v] = freqs.inv[i + v];
  const float g = static_cast<float>(gain);
  // launched as a programmatic dependent of what precedes it, as the plain
  // table is: nothing is read or written before that grid has finished
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (long long r = blockIdx.x * (long long)rows_per_block + threadIdx.x / per_row; r < n_rows;
       r += (long long)gridDim.x * rows_per_block) {
    const double p = static_cast<double>(pos[r]);
    float c[VEC], s[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const double angle = p * inv[v];
      if (fabs(angle) < 1099511627776.0) {  // 2^40
        sincos_reduced(angle, s[v], c[v]);
        c[v] *= g;
        s[v] *= g;
      } else {
        double sd, cd;
        sincos(angle, &sd, &cd);
        c[v] = static_cast<float>(cd * gain);
        s[v] = static_cast<float>(sd * gain);
      }
    }
    float* co = cos_out + r * 2 * half + i;
    float* so = sin_out + r * 2 * half + i;
    if constexpr (VEC == 4) {
      const float4 cv = make_float4(c[0], c[1], c[2], c[3]), sv = make_float4(s[0], s[1], s[2], s[3]);
      if (stream_out) {
        __stcs(reinterpret_cast<float4*>(co), cv);
        __stcs(reinterpret_cast<float4*>(co + half), cv);
        __stcs(reinterpret_cast<float4*>(so), sv);
        __stcs(reinterpret_cast<float4*>(so + half), sv);
      } else {
        *reinterpret_cast<float4*>(co) = cv;
        *reinterpret_cast<float4*>(co + half) = cv;
        *reinterpret_cast<float4*>(so) = sv;
        *reinterpret_cast<float4*>(so + half) = sv;
      }
    } else {
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        co[v] = c[v];
        co[v + half] = c[v];
        so[v] = s[v];
        so[v + half] = s[v];
      }
    }
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
  int blocks[2];     // vector kernel: head blocks of q and k
};

__device__ __forceinline__ float ra_load(const float* p) { return *p; }
__device__ __forceinline__ float ra_load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void ra_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void ra_store(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// 16 bytes of a head: its elements as floats, and back with one rounding.
__device__ __forceinline__ void ra_unpack(const uint4& u, float (&f)[8]) {
  f[0] = bf16lo(u.x), f[1] = bf16hi(u.x), f[2] = bf16lo(u.y), f[3] = bf16hi(u.y);
  f[4] = bf16lo(u.z), f[5] = bf16hi(u.z), f[6] = bf16lo(u.w), f[7] = bf16hi(u.w);
}
__device__ __forceinline__ void ra_unpack(const uint4& u, float (&f)[4]) {
  f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y);
  f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ uint4 ra_pack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 ra_pack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}

// Whole 16-byte chunks: a thread takes one chunk position of HB heads of a
// token -- with its partner chunk R/2 further on in the half layout -- so that
// the table's values are read once for HB heads and HB or 2 HB loads are in
// flight; the lanes of a warp run over a head's chunks first, so each load is
// of whole lines.  Chunks from R on are copied (unless in place).  Bound by
// reading and writing x.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(ra::THREADS) rope_apply_vec_kernel(RopeApplyParams p) {
  constexpr int VE = 16 / sizeof(T);
  constexpr int HB = ra::HB;
  const int half = p.R / 2;
  const int rot = (INTERLEAVED ? p.R : half) / VE;  // chunks (or pairs of chunks) that turn
  const int units = rot + (p.D - p.R) / VE;
  const int n_blk = p.blocks[0] + p.blocks[1];
  const long long total = p.tokens * n_blk * units;
  const long long idx = blockIdx.x * (long long)ra::THREADS + threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (idx >= total) return;
  long long tok;
  int rest;
  if (total <= 0xffffffffLL) {  // (32-bit division is a fraction of the 64-bit one)
    const unsigned per = static_cast<unsigned>(n_blk) * units;
    const unsigned t = static_cast<unsigned>(idx) / per;
    tok = t;
    rest = static_cast<int>(static_cast<unsigned>(idx) - t * per);
  } else {
    const long long per = static_cast<long long>(n_blk) * units;
    tok = idx / per;
    rest = static_cast<int>(idx - tok * per);
  }
  int blk = rest / units;
  const int u = rest - blk * units;
  const bool is_k = blk >= p.blocks[0];
  const RopeSide& sd = p.side[is_k];
  if (is_k) blk -= p.blocks[0];
  const int b = static_cast<int>(tok) / p.seq, s = static_cast<int>(tok) - b * p.seq;
  const T* x = static_cast<const T*>(sd.x) + b * sd.xb + s * sd.xs + blk * HB * sd.xh;
  T* y = static_cast<T*>(sd.y) + b * sd.yb + s * sd.ys + blk * HB * sd.yh;
  const int n = min(HB, sd.heads - blk * HB);
  if (u >= rot) {
    if (sd.x == sd.y) return;
    const int d = p.R + (u - rot) * VE;
    uint4 v[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j)
      if (j < n) v[j] = *reinterpret_cast<const uint4*>(x + j * sd.xh + d);
#pragma unroll
    for (int j = 0; j < HB; ++j)
      if (j < n) *reinterpret_cast<uint4*>(y + j * sd.yh + d) = v[j];
    return;
  }
  const int d = u * VE;
  if constexpr (INTERLEAVED) {
    constexpr int NP = VE / 2;  // pairs of a chunk
    uint4 v[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j)
      if (j < n) v[j] = *reinterpret_cast<const uint4*>(x + j * sd.xh + d);
    float c[NP], sn[NP];
    const float* cr = p.cos + tok * p.R + d / 2;
    const float* sr = p.sin + tok * p.R + d / 2;
#pragma unroll
    for (int e = 0; e < NP; e += 2) {
      const float2 cv = *reinterpret_cast<const float2*>(cr + e);
      const float2 sv = *reinterpret_cast<const float2*>(sr + e);
      c[e] = cv.x, c[e + 1] = cv.y;
      sn[e] = p.sign * sv.x, sn[e + 1] = p.sign * sv.y;
    }
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      if (j < n) {
        float f[VE];
        ra_unpack(v[j], f);
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          const float a = f[2 * e], z = f[2 * e + 1];
          f[2 * e] = fmaf(a, c[e], -z * sn[e]);
          f[2 * e + 1] = fmaf(z, c[e], a * sn[e]);
        }
        *reinterpret_cast<uint4*>(y + j * sd.yh + d) = ra_pack(f);
      }
    }
  } else {
    uint4 v[HB], w[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j)
      if (j < n) {
        v[j] = *reinterpret_cast<const uint4*>(x + j * sd.xh + d);
        w[j] = *reinterpret_cast<const uint4*>(x + j * sd.xh + d + half);
      }
    float c[VE], sn[VE];
    const float* cr = p.cos + tok * p.R + d;
    const float* sr = p.sin + tok * p.R + d;
#pragma unroll
    for (int e = 0; e < VE; e += 4) {
      const float4 cv = *reinterpret_cast<const float4*>(cr + e);
      const float4 sv = *reinterpret_cast<const float4*>(sr + e);
      c[e] = cv.x, c[e + 1] = cv.y, c[e + 2] = cv.z, c[e + 3] = cv.w;
      sn[e] = p.sign * sv.x, sn[e + 1] = p.sign * sv.y;
      sn[e + 2] = p.sign * sv.z, sn[e + 3] = p.sign * sv.w;
    }
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      if (j < n) {
        float a[VE], z[VE];
        ra_unpack(v[j], a);
        ra_unpack(w[j], z);
#pragma unroll
        for (int e = 0; e < VE; ++e) {
          const float ya = fmaf(a[e], c[e], -z[e] * sn[e]);
          z[e] = fmaf(z[e], c[e], a[e] * sn[e]);
          a[e] = ya;
        }
        *reinterpret_cast<uint4*>(y + j * sd.yh + d) = ra_pack(a);
        *reinterpret_cast<uint4*>(y + j * sd.yh + d + half) = ra_pack(z);
      }
    }
  }
}

// Any even R, any alignment and strides: a thread per pair or per copied element,
// three 64-bit divisions and narrow accesses for each, so far from what its bytes
// would take: 8192 tokens of 72 heads in bf16, D 96 / R 24 334 us (bytes: 35), D 80
// / R 20 284 (29), D 80 / R 40 257 (29); in fp32, D 80 / R 20 283 (58).
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(ra::THREADS) rope_apply_any_kernel(RopeApplyParams p) {
  const int half = p.R / 2;
  const int per_head = half + (p.D - p.R);
  const long long heads = p.side[0].heads + p.side[1].heads;
  const long long total = p.tokens * heads * per_head;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
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
