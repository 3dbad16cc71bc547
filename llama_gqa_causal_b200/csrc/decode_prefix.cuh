// Decode for a batch whose sequences share a prefix: one query row per head
// against the prefix's rows and the sequence's own rows, in one softmax.
//
// For a K/V head the query rows of the whole batch (bsz x group of them) meet
// the same prefix, so that part is a product of matrices and runs on tcgen05:
//   S = Q K_prefix^T (128 query rows x 128 keys), P = 2^(S c - m), O += P V_prefix
// with each prefix tile read once for up to 256 query rows.  The sequences' own
// rows are read once each by decode_share, the split-KV decode.  Both parts run
// in one launch of one CTA per SM: the CTAs are dealt out on the device, in
// proportion to the two parts' work (cache_lens is known only there), because
// the prefix part is bound by exponentials and products as soon as a few rows
// share a tile, and the own part by memory.  decode_prefix_combine_kernel
// merges the partials of both by the log-sum-exp identity
//   m* = max_s m_s,  l = sum_s l_s 2^(m_s - m*),  o = sum_s o_s 2^(m_s - m*) / l.
//
// Prefix work is a list of items, an item being 128 keys against a tile pair
// (256 query rows of one K/V head, as two units of 128), in the order
// (tile pair, K/V head, keys).  A CTA takes a contiguous run of items; each run
// inside one (tile pair, K/V head) is a segment and leaves one partial per
// unit.  If the tile pair holds at most 128 rows, both units work on the same
// rows and take the key tiles in turn, so that one unit's softmax still runs
// beside the other's products.
//
// Warp roles of a prefix CTA (384 threads = three warpgroups): warp 0 TMA
// producer (one ring of K and V tiles in the order of their use), warp 1 TMEM
// and MMA issuer, warps 4-7 and 8-11 the softmax of unit 0 and 1 (a thread per
// query row = TMEM lane).  TMEM: S_0, S_1 (128 columns each; P overwrites S),
// O_0, O_1 (D each).
#pragma once
#include <type_traits>

#include "decode_bf16.cuh"

namespace la {
namespace px {
constexpr int BM = 128;      // query rows of a unit (= TMEM lanes)
constexpr int BN = 128;      // keys of a tile
constexpr int THREADS = 384;
constexpr int MAX_CTAS = 148;
// Ring of K and V tiles: what fits beside two Q tiles.
__host__ __device__ constexpr int ring(int d) { return d == 128 ? 5 : 10; }
// The split of 384 x 168 registers: 56 + 224 + 224 a lane.
constexpr int kRegsControl = 56;
constexpr int kRegsSoftmax = 224;
constexpr int kRegsAtLaunch = (65536 / THREADS) / 8 * 8;  // 168
static_assert(kRegsControl % 8 == 0 && kRegsSoftmax % 8 == 0, "setmaxnreg takes multiples of 8");
static_assert(kRegsControl + 2 * kRegsSoftmax <= 3 * kRegsAtLaunch,
              "setmaxnreg split exceeds the registers the block is launched with");
constexpr float kRescaleThreshold = 8.0f;  // log2 units
constexpr int kPolyPairsOf8 = 3;  // pairs of 8 exponentiated on the FMA pipe
// Work of an item and of a 64-row chunk of a cache, in units that only their
// ratios matter of: what one SM takes for it.
__host__ __device__ constexpr float cost_pair(int d) { return d == 128 ? 2.1f : 1.5f; }
__host__ __device__ constexpr float cost_single(int d) { return d == 128 ? 1.2f : 0.8f; }
__host__ __device__ constexpr float cost_chunk(int d) { return d == 128 ? 0.55f : 0.35f; }
// Floats of one unit's partial: [D + 2][BM], the outputs of a row down a
// column, then its maximum and sum (lanes are rows, so both the writing warp
// and the combining one touch whole lines).
__host__ __device__ constexpr int unit_floats(int d) { return (d + 2) * BM; }
constexpr int HDR = 4;  // ints before the chunk prefix: groups, CTAs of a group, own CTAs
}  // namespace px

struct PrefixParams {
  const __nv_bfloat16* q;  // [b, H, D]
  float* part;             // [tile pairs * Hkv + MAX_CTAS][2][D + 2][BM]
  int* hdr;                // [HDR + b + 1]
  int rows;                // query rows of a K/V head: b * group
  int P;                   // keys
  int nt;                  // key tiles
  int pairs;               // tile pairs: ceil(rows / 256)
  int H, Hkv, group;
  float scale_log2;
};

// How the CTAs are dealt out.  The prefix's items are split over groups of
// `per` CTAs: one group per tile pair, so that the CTAs of different tile pairs
// read the same keys at about the same time, or one group for everything where
// whole groups would leave more than an eighth of the prefix's CTAs idle.
struct PrefixPlan {
  int groups, per, own;
};
__device__ __forceinline__ PrefixPlan prefix_plan(const PrefixParams& x, long long n_chunks,
                                                  int n_ctas, float c_pair, float c_single,
                                                  float c_chunk) {
  PrefixPlan r = {0, 0, 0};
  const long long items = static_cast<long long>(x.Hkv) * x.nt;  // of one tile pair
  if (items > 0) {
    const bool single = x.rows - (x.pairs - 1) * 2 * px::BM <= px::BM;  // the last pair
    const float wa = static_cast<float>(items) *
                     (static_cast<float>(x.pairs - single) * c_pair + (single ? c_single : 0.f));
    const float wb = static_cast<float>(n_chunks) * c_chunk;
    int na = static_cast<int>(static_cast<float>(n_ctas) * wa / (wa + wb) + 0.5f);
    na = max(1, min(na, n_chunks > 0 ? n_ctas - 1 : n_ctas));
    if (x.pairs <= na && (na / x.pairs) * x.pairs * 8 >= na * 7) {
      r.groups = x.pairs;
      r.per = static_cast<int>(min(static_cast<long long>(na / x.pairs), items));
    } else {
      r.groups = 1;
      r.per = static_cast<int>(min(static_cast<long long>(na), items * x.pairs));
    }
  }
  r.own = static_cast<int>(min(n_chunks, static_cast<long long>(n_ctas - r.groups * r.per)));
  return r;
}

template <int D>
struct PrefixSmem {
  alignas(1024) __nv_bfloat16 q[2][px::BM * D];
  alignas(1024) __nv_bfloat16 ring[px::ring(D)][px::BN * D];
  uint64_t full[px::ring(D)], empty[px::ring(D)];
  uint64_t q_ready[2], s_full[2], p_lo[2], p_hi[2], o_full[2];
  uint64_t mma_done;
  uint32_t tmem_base;
};

// Maximum that a NaN operand makes NaN.
__device__ __forceinline__ float fmax3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// 2^x for a pair on the FMA and integer pipes, as exp2_poly2 but with a cubic
// for 2^f (largest relative error 7.5e-5, far below the 2^-9 that rounding the
// result to bf16 may cost; csrc/fit_exp2_poly.py with degree 3).
__device__ __forceinline__ void exp2_cubic2(float& y0, float& y1, float x0, float x1) {
  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23
  constexpr float c0 = 0.9999280571937561f, c1 = 0.6932609677314758f;
  constexpr float c2 = 0.2426111251115799f, c3 = 0.0551716685295105f;
  x0 = fmaxf(x0, -126.f);
  x1 = fmaxf(x1, -126.f);
  float t0, t1, n0, n1, f0, f1, q0, q1;
  fadd2(t0, t1, x0, x1, kRound, kRound);      // round(x) in the low bits of t
  fadd2(n0, n1, t0, t1, -kRound, -kRound);    // n = round(x) as a float
  ffma2(f0, f1, n0, n1, -1.f, -1.f, x0, x1);  // f = x - n
  ffma2(q0, q1, c3, c3, f0, f1, c2, c2);
  ffma2(q0, q1, q0, q1, f0, f1, c1, c1);
  ffma2(q0, q1, q0, q1, f0, f1, c0, c0);
  y0 = __int_as_float(__float_as_int(q0) + (__float_as_int(t0) << 23));
  y1 = __int_as_float(__float_as_int(q1) + (__float_as_int(t1) << 23));
}

// A run of items inside one (tile pair, K/V head).
struct PrefixSegment {
  int seq, kvh;   // seq = tile pair * Hkv + kvh
  int row0, rows; // of the K/V head's query rows
  int j0, n;      // key tiles
  bool single;    // both units on the same rows, key tiles in turn
};
__device__ __forceinline__ PrefixSegment prefix_segment(const PrefixParams& x, long long i0,
                                                        long long i1) {
  PrefixSegment g;
  const long long seq = i0 / x.nt;
  g.seq = static_cast<int>(seq);
  g.j0 = static_cast<int>(i0 - seq * x.nt);
  g.n = static_cast<int>(min(static_cast<long long>(x.nt - g.j0), i1 - i0));
  const int pair = g.seq / x.Hkv;
  g.kvh = g.seq - pair * x.Hkv;
  g.row0 = pair * 2 * px::BM;
  g.rows = min(2 * px::BM, x.rows - g.row0);
  g.single = g.rows <= px::BM;
  return g;
}

// The items [x0, x1) by one CTA.
template <int D>
__device__ __forceinline__ void prefix_share(PrefixSmem<D>& s, const CUtensorMap& tm_k,
                                             const CUtensorMap& tm_v, const PrefixParams& x,
                                             int cta, long long x0, long long x1) {
  using namespace px;
  constexpr int CB = D / 64;                  // 64-column swizzle blocks per row
  constexpr int NST = ring(D);
  constexpr uint32_t BLOCK_BYTES = BM * 128;  // one [128 rows x 64 cols] bf16 block
  constexpr uint32_t TILE_BYTES = BM * D * 2;
  constexpr uint32_t IDESC_QK = idesc_bf16(BM, BN, false);
  constexpr uint32_t IDESC_PV = idesc_bf16(BM, D, true);
  constexpr uint32_t TMEM_COLS = 512;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < NST; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&s.q_ready[t], 4);
      mbar_init(&s.s_full[t], 1);
      mbar_init(&s.p_lo[t], 4);
      mbar_init(&s.p_hi[t], 4);
      mbar_init(&s.o_full[t], 1);
    }
    mbar_init(&s.mma_done, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&s.tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  fence_proxy_async_smem();  // the chunk scan wrote where the ring's copies land
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  auto tm_s = [&](int t) { return tmem + static_cast<uint32_t>(t * BN); };
  auto tm_o = [&](int t) { return tmem + static_cast<uint32_t>(2 * BN + t * D); };

  if (warp == 0) {
    // ================================================================ TMA producer
    // Tiles in the order of their use: of a segment K_0 (and K_1 if the units
    // take the tiles in turn), then V_j and the K tile that follows the ones sent.
    setmaxnreg_dec<kRegsControl>();
    if (elect_one()) {
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
    __syncwarp();
    uint32_t sent = 0;  // tiles put into the ring
    bool ok = true;
    auto send = [&](const CUtensorMap* m, int kvh, int j) {
      const int st = static_cast<int>(sent % NST);
      if (sent >= NST && !mbar_wait(&s.empty[st], (sent / NST - 1) & 1)) {
        ok = false;
        return;
      }
      if (elect_one()) {
        mbar_arrive_expect_tx(&s.full[st], TILE_BYTES);
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
          tma_load_3d(reinterpret_cast<uint8_t*>(&s.ring[st][0]) + cb * BLOCK_BYTES, m, &s.full[st],
                      cb * 64, j * BN, kvh);
      }
      __syncwarp();
      ++sent;
    };
    for (long long i = x0; i < x1 && ok;) {
      const PrefixSegment g = prefix_segment(x, i, x1);
      i += g.n;
      const int ahead = g.single ? 2 : 1;
      send(&tm_k, g.kvh, g.j0);
      if (g.single && g.n > 1 && ok) send(&tm_k, g.kvh, g.j0 + 1);
      for (int j = 0; j < g.n && ok; ++j) {
        send(&tm_v, g.kvh, g.j0 + j);
        if (ok && j + ahead < g.n) send(&tm_k, g.kvh, g.j0 + j + ahead);
      }
    }
    // leave no copy in flight
    for (uint32_t i = sent > NST ? sent - NST : 0; i < sent; ++i)
      if (!mbar_wait(&s.full[i % NST], (i / NST) & 1)) break;
  } else if (warp == 1) {
    // ================================================================ MMA issuer
    setmaxnreg_dec<kRegsControl>();
    const uint64_t q_desc0 = sw128_desc(smem_u32(&s.q[0][0]), 16, 1024);
    const uint64_t k_desc0 = sw128_desc(smem_u32(&s.ring[0][0]), 16, 1024);
    const uint64_t v_desc0 = sw128_desc(smem_u32(&s.ring[0][0]), BLOCK_BYTES, 1024);
    auto issue_qk = [&](int t, int tq, int st) {  // S_t = Q_tq K^T
      const uint64_t qd = q_desc0 + ((static_cast<uint32_t>(tq) * TILE_BYTES) >> 4);
      const uint64_t kd = k_desc0 + ((static_cast<uint32_t>(st) * TILE_BYTES) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk / 4) * BLOCK_BYTES + (kk % 4) * 32) >> 4;
          mma_ss(tm_s(t), qd + off, kd + off, IDESC_QK, kk > 0 ? 1u : 0u);
        }
        tc_commit(&s.s_full[t]);
      }
      __syncwarp();
    };
    auto issue_pv = [&](int t, int st, bool accumulate, int h) {  // keys [64h, 64h + 64)
      const uint64_t vd = v_desc0 + ((static_cast<uint32_t>(st) * TILE_BYTES) >> 4);
      if (elect_one()) {
#pragma unroll
        for (int kk = h * (BN / 32); kk < (h + 1) * (BN / 32); ++kk)
          mma_ts(tm_o(t), tm_s(t) + kk * 8, vd + ((kk * 2048) >> 4), IDESC_PV,
                 (accumulate || kk > h * (BN / 32)) ? 1u : 0u);
      }
      __syncwarp();
    };
    auto commit = [&](uint64_t* bar) {
      if (elect_one()) tc_commit(bar);
      __syncwarp();
    };
    uint32_t used = 0;  // tiles taken from the ring
    uint32_t cnt[2] = {0, 0};  // P tiles of each unit so far
    uint32_t seg = 0;
    bool ok = true;
    auto wait_tile = [&](uint32_t i) {
      ok = mbar_wait(&s.full[i % NST], (i / NST) & 1);
      if (ok) tc_fence_after();
      return ok;
    };
    auto half = [&](int t, int st, bool accumulate, int h) {
      if (!mbar_wait(h ? &s.p_hi[t] : &s.p_lo[t], cnt[t] & 1)) return false;
      tc_fence_after();
      issue_pv(t, st, accumulate, h);
      return true;
    };
    for (long long i = x0; i < x1 && ok; ++seg) {
      const PrefixSegment g = prefix_segment(x, i, x1);
      i += g.n;
      ok = mbar_wait(&s.q_ready[0], seg & 1) && mbar_wait(&s.q_ready[1], seg & 1);
      if (!ok || !wait_tile(used)) break;
      if (g.single) {
        issue_qk(0, 0, static_cast<int>(used % NST));
        commit(&s.empty[used % NST]);
        ++used;
        if (g.n > 1) {
          if (!wait_tile(used)) break;
          issue_qk(1, 0, static_cast<int>(used % NST));
          commit(&s.empty[used % NST]);
          ++used;
        }
        for (int j = 0; j < g.n; ++j) {
          const int t = j & 1;
          const int vs = static_cast<int>(used % NST);
          if (!wait_tile(used)) break;
          ++used;
          ok = half(t, vs, j > 1, 0) && half(t, vs, true, 1);
          if (!ok) break;
          ++cnt[t];
          commit(&s.empty[vs]);
          if (j + 2 < g.n) {
            if (!wait_tile(used)) break;
            issue_qk(t, 0, static_cast<int>(used % NST));
            commit(&s.empty[used % NST]);
            ++used;
          } else {
            commit(&s.o_full[t]);
          }
        }
        // (a unit without a tile waits here all the same: running ahead, it would
        // complete two phases of q_ready between two of this warp's waits)
        if (ok && g.n == 1) commit(&s.o_full[1]);
      } else {
        issue_qk(0, 0, static_cast<int>(used % NST));
        issue_qk(1, 1, static_cast<int>(used % NST));
        commit(&s.empty[used % NST]);
        ++used;
        for (int j = 0; j < g.n && ok; ++j) {
          const bool next = j + 1 < g.n;
          const int vs = static_cast<int>(used % NST);
          const uint32_t kn = used + 1;
          if (!wait_tile(used)) break;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            ok = half(t, vs, j > 0, 0) && half(t, vs, true, 1);
            if (!ok) break;
            ++cnt[t];
            if (next) {
              if (t == 0 && !wait_tile(kn)) break;
              issue_qk(t, t, static_cast<int>(kn % NST));
            } else {
              commit(&s.o_full[t]);
            }
          }
          if (!ok) break;
          commit(&s.empty[vs]);
          if (next) commit(&s.empty[kn % NST]);
          used = next ? kn + 1 : kn;
        }
      }
    }
    // every MMA this warp issued has completed before the CTA can exit
    commit(&s.mma_done);
    mbar_wait(&s.mma_done, 0);
  } else if (warp < 4) {
    setmaxnreg_dec<kRegsControl>();  // idle warps of warpgroup 0
  } else {
    // ================================================================ softmax
    setmaxnreg_inc<kRegsSoftmax>();
    const int t = (warp - 4) >> 2;
    const int quarter = warp & 3;
    const int r = quarter * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t my_s = tm_s(t) + lane_off, my_o = tm_o(t) + lane_off;
    const float c_log2 = x.scale_log2;
    const bool scale_pos = c_log2 > 0.f;
    uint32_t sc = 0, oc = 0;  // S tiles and finished segments of this unit so far
    bool ok = true;
    for (long long i = x0; i < x1 && ok;) {
      const PrefixSegment g = prefix_segment(x, i, x1);
      i += g.n;
      const int tq = g.single ? 0 : t;
      const int rows = min(BM, g.rows - tq * BM);  // of this unit
      const bool active = quarter * 32 < rows;     // (warps past the rows only keep step)
      // ---- Q rows into the unit's tile: row m of the K/V head is batch entry
      // m / group, head kvh * group + m % group; a row's 16-byte chunks go to
      // adjacent lanes.  Rows past the end are zero.
      if (tq == t) {
        constexpr int CH16 = D / 8;
        constexpr int RPS = 32 / CH16;
        uint4 v[32 / RPS];
#pragma unroll
        for (int st = 0; st < 32 / RPS; ++st) {
          const int rr = quarter * 32 + st * RPS + lane / CH16;
          v[st] = make_uint4(0, 0, 0, 0);
          if (rr < rows) {
            const int m = g.row0 + tq * BM + rr;
            const int b = m / x.group, h = m - b * x.group;
            v[st] = *reinterpret_cast<const uint4*>(
                x.q + (static_cast<size_t>(b) * x.H + g.kvh * x.group + h) * D + (lane % CH16) * 8);
          }
        }
        uint8_t* qs = reinterpret_cast<uint8_t*>(&s.q[t][0]);
#pragma unroll
        for (int st = 0; st < 32 / RPS; ++st) {
          const int rr = quarter * 32 + st * RPS + lane / CH16;
          const int c = lane % CH16;
          *reinterpret_cast<uint4*>(qs + (c / 8) * BLOCK_BYTES + sw128_offset(rr, c % 8)) = v[st];
        }
        fence_proxy_async_smem();
      }
      tc_fence_before();  // (the last segment's O has been read)
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_ready[t]);

      float m_ref = -INFINITY;  // reference maximum (log2 units) of the exponentials
      float l_sum = 0.f;
      const int n_mine = g.single ? (g.n + 1 - t) / 2 : g.n;
      for (int jj = 0; jj < n_mine; ++jj) {
        const int j = g.j0 + (g.single ? 2 * jj + t : jj);
        if (!mbar_wait(&s.s_full[t], sc & 1)) { ok = false; break; }
        ++sc;
        tc_fence_after();
        if (!active) {
          if (lane == 0) {
            mbar_arrive(&s.p_lo[t]);
            mbar_arrive(&s.p_hi[t]);
          }
          __syncwarp();
          continue;
        }
        uint32_t sr[4][32];
        tmem_ld32(my_s, sr[0]);
        tmem_ld32(my_s + 32, sr[1]);
        tmem_ld_wait(sr[0]);
        tmem_ld_wait(sr[1]);
        tmem_ld32(my_s + 64, sr[2]);
        tmem_ld32(my_s + 96, sr[3]);
        // raw scores (the scale is folded into the exponent's FMA), or scaled
        // and masked ones: the last tile's keys past the end, and any tile if
        // the scale is not positive (the maximum is then another key's)
        const int left = x.P - j * BN;  // keys of this tile and after it
        auto tile = [&](auto edge_c) {
          constexpr bool kEdge = decltype(edge_c)::value;
          float v[BN];
          auto fill = [&](int e0) {
#pragma unroll
            for (int e = e0; e < e0 + BN / 2; ++e) {
              const float raw = __uint_as_float(sr[e / 32][e % 32]);
              v[e] = !kEdge ? raw : e < left ? raw * c_log2 : -INFINITY;
            }
          };
          float mm[8];
          fill(0);
#pragma unroll
          for (int k = 0; k < 8; ++k) mm[k] = fmax3_nan(v[k], v[k + 8], v[k + 8]);
#pragma unroll
          for (int e = 16; e < BN / 2; e += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) mm[k] = fmax3_nan(mm[k], v[e + k], v[e + k + 8]);
          tmem_ld_wait(sr[2]);
          tmem_ld_wait(sr[3]);
          fill(BN / 2);
#pragma unroll
          for (int e = BN / 2; e < BN; e += 16)
#pragma unroll
            for (int k = 0; k < 8; ++k) mm[k] = fmax3_nan(mm[k], v[e + k], v[e + k + 8]);
          float mx = fmax3_nan(fmax3_nan(mm[0], mm[1], mm[2]), fmax3_nan(mm[3], mm[4], mm[5]),
                               fmax3_nan(mm[6], mm[7], mm[7]));
          if (!kEdge) mx *= c_log2;
          // lazy reference: moved only when the maximum grows by more than the
          // threshold; a NaN score makes the reference, and with it the row, NaN
          float alpha = 1.f;
          if (!(mx <= m_ref + kRescaleThreshold)) {
            alpha = (m_ref == -INFINITY) ? 0.f : ex2_approx(m_ref - mx);
            m_ref = mx;
          }
          const float nref = (m_ref == -INFINITY) ? 0.f : -m_ref;
          const float cc = kEdge ? 1.f : c_log2;
          float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          // P in two halves: the product with V starts on the first while the
          // second is exponentiated; part of that hides the first's store
          uint32_t pk[2][32];
          auto exps = [&](int e0, int e1) {
#pragma unroll
            for (int e = e0; e < e1; e += 2) {
              float a0, a1, p0, p1;
              ffma2(a0, a1, v[e], v[e + 1], cc, cc, nref, nref);
              if (!kEdge && ((e / 2) % 8) < kPolyPairsOf8) {
                exp2_cubic2(p0, p1, a0, a1);
              } else {
                p0 = ex2_approx(a0);
                p1 = ex2_approx(a1);
              }
              const int k = (e / 2) % 4;
              fadd2(acc[2 * k], acc[2 * k + 1], acc[2 * k], acc[2 * k + 1], p0, p1);
              // rounded to bf16 as the tensor cores take it; the sum is of the
              // unrounded values
              pk[e / 64][(e % 64) / 2] = pack_bf16x2(p0, p1);
            }
          };
          auto release = [&](uint64_t* bar) {
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar);
          };
          exps(0, 64);
          if (jj > 0 && __any_sync(0xffffffffu, !(alpha == 1.f))) {
            // O is corrected before any P of this tile is released; the product
            // of the unit's last tile has completed (committed before this S)
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t orr[32];
              tmem_ld32(my_o + c * 32, orr);
              tmem_ld_wait(orr);
#pragma unroll
              for (int e = 0; e < 32; ++e) orr[e] = __float_as_uint(__uint_as_float(orr[e]) * alpha);
              tmem_st32(my_o + c * 32, orr);
            }
          }
          tmem_st32(my_s, pk[0]);
          exps(64, 80);
          release(&s.p_lo[t]);
          exps(80, 128);
          tmem_st32(my_s + 32, pk[1]);
          release(&s.p_hi[t]);
          l_sum = fmaf(l_sum, alpha, ((acc[0] + acc[1]) + (acc[2] + acc[3])) +
                                         ((acc[4] + acc[5]) + (acc[6] + acc[7])));
        };
        if (left < BN || !scale_pos) tile(std::true_type{});
        else tile(std::false_type{});
      }
      if (!ok) break;
      // ---- the segment's partial of this unit
      const int slot = g.j0 == 0 ? g.seq : x.pairs * x.Hkv + cta;
      float* dst = x.part + (static_cast<size_t>(slot) * 2 + t) * unit_floats(D) + r;
      if (!mbar_wait(&s.o_full[t], oc & 1)) break;
      ++oc;
      tc_fence_after();
      if (active && n_mine > 0) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t orr[32];
          tmem_ld32(my_o + c * 32, orr);
          tmem_ld_wait(orr);
          if (r < rows)
#pragma unroll
            for (int e = 0; e < 32; ++e) dst[(c * 32 + e) * BM] = __uint_as_float(orr[e]);
        }
      }
      if (r < rows) {
        dst[D * BM] = m_ref;
        dst[(D + 1) * BM] = l_sum;
      }
      __syncwarp();
    }
  }

  // ---- teardown
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TMEM_COLS);
  }
}

template <int D>
constexpr size_t prefix_smem_bytes() {
  return (sizeof(PrefixSmem<D>) > sizeof(DecSmem<D>) ? sizeof(PrefixSmem<D>) : sizeof(DecSmem<D>)) +
         1024;
}

template <int D, bool APPEND>
__global__ void __launch_bounds__(px::THREADS, 1)
    decode_prefix_kernel(const __grid_constant__ CUtensorMap tm_kp,
                         const __grid_constant__ CUtensorMap tm_vp,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v, PrefixParams x, DecodeParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  DecSmem<D>& own = *reinterpret_cast<DecSmem<D>*>(smem);
  // a programmatic dependent of what precedes it: no global memory before this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  scan_chunks<APPEND, px::THREADS>(own.chunk_prefix, p);
  const long long n_chunks = static_cast<long long>(own.chunk_prefix[p.bsz]) * p.Hkv * p.hchunks;
  const PrefixPlan plan = prefix_plan(x, n_chunks, gridDim.x, px::cost_pair(D), px::cost_single(D),
                                      px::cost_chunk(D));
  if (blockIdx.x == 0) {  // for the combine kernel
    if (threadIdx.x == 0) {
      x.hdr[0] = plan.groups;
      x.hdr[1] = plan.per;
      x.hdr[2] = plan.own;
    }
    for (int b = threadIdx.x; b <= p.bsz; b += px::THREADS) p.ws_prefix[b] = own.chunk_prefix[b];
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int cta = blockIdx.x, n_prefix = plan.groups * plan.per;
  if (cta < n_prefix) {
    const long long items = static_cast<long long>(x.Hkv) * x.nt * (x.pairs / plan.groups);
    const int group = cta / plan.per, i = cta - group * plan.per;
    __syncthreads();  // the scan's shared memory is free: CTA 0 has read it
    prefix_share<D>(*reinterpret_cast<PrefixSmem<D>*>(smem), tm_kp, tm_vp, x, cta,
                    group * items + share_start(i, items, plan.per),
                    group * items + share_start(i + 1, items, plan.per));
    return;
  }
  if (cta - n_prefix >= plan.own) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < dec::NSTAGE; ++i) {
      mbar_init(&own.full[i], 1);
      mbar_init(&own.empty[i], dec::NCW);
    }
    fence_mbar_init();
  }
  __syncthreads();
  if (threadIdx.x >= dec::THREADS) return;
  decode_share<D, APPEND>(own, tm_k, tm_v, p, cta - n_prefix, plan.own);
}

// Merges the partials of 32 query rows of one K/V head, 8 dimensions a block:
// a lane is a row, and the eight warps take the partials in turn (a short batch
// behind a long prefix has over a hundred of them) and are merged through
// shared memory.
namespace px {
constexpr int COMBINE_WARPS = 8;
}
template <int D>
__global__ void __launch_bounds__(px::COMBINE_WARPS * 32)
    decode_prefix_combine_kernel(PrefixParams x, DecodeParams p, __nv_bfloat16* __restrict__ out) {
  using namespace px;
  constexpr int DC = D / 8;
  constexpr int W = COMBINE_WARPS;
  __shared__ float so[W][8][33], sm[W][33], sl[W][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int d0 = static_cast<int>(blockIdx.x % DC) * 8;
  const int rb = static_cast<int>(blockIdx.x / DC);
  const int blocks_per_kvh = (x.rows + 31) / 32;
  const int kvh = rb / blocks_per_kvh;
  const int row0 = (rb - kvh * blocks_per_kvh) * 32;
  const int row = row0 + lane;
  const bool valid = row < x.rows;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int groups = x.hdr[0], per = x.hdr[1], n_own = x.hdr[2];
  float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
  auto add = [&](float mc, float lc, const float (&oc)[8]) {
    if (lc == 0.f) return;  // (no weight in it; a NaN sum is not 0 and stays)
    const float m_new = fmax3_nan(m, mc, mc);
    const float fo = m == -INFINITY ? 0.f : ex2_approx(m - m_new);
    const float fc = ex2_approx(mc - m_new);
    l = l * fo + lc * fc;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = o[e] * fo + oc[e] * fc;
    m = m_new;
  };

  // ---- prefix partials: the home slot, then those of the CTAs whose run starts
  // inside this (tile pair, K/V head); two units each if they share their rows
  int taken = 0;  // partials dealt out to the warps so far
  if (groups > 0) {
    const int pair = row0 / (2 * BM), in_pair = row0 - pair * 2 * BM;
    const bool single = x.rows - pair * 2 * BM <= BM;
    const int seq = pair * x.Hkv + kvh;
    const long long first = static_cast<long long>(seq) * x.nt;
    const long long items = static_cast<long long>(x.Hkv) * x.nt * (x.pairs / groups);
    const long long group = first / items, at = first - group * items;
    const int c0 = static_cast<int>(group * per + share_owner(at, items, per));
    const int c1 = static_cast<int>(group * per + share_owner(at + x.nt - 1, items, per));
    const int n = (c1 - c0 + 1) << single;
    for (int k = warp; k < n; k += W) {
      const int seg = k >> single;
      const int unit = single ? k & 1 : in_pair / BM;
      const int slot = seg == 0 ? seq : x.pairs * x.Hkv + c0 + seg;
      const float* src = x.part + (static_cast<size_t>(slot) * 2 + unit) * unit_floats(D) +
                         in_pair % BM + lane;
      if (valid) {
        float oc[8];
        const float mc = src[D * BM], lc = src[(D + 1) * BM];
#pragma unroll
        for (int e = 0; e < 8; ++e) oc[e] = src[(d0 + e) * BM];
        add(mc, lc, oc);
      }
    }
    taken = n;
  }
  // ---- the sequence's own partials, laid out as decode_share writes them
  if (valid) {
    const int b = row / x.group, h = row - b * x.group;
    const int hc = h / 8;
    const long long before = p.ws_prefix[b];
    const int nch = static_cast<int>(p.ws_prefix[b + 1] - before);
    if (nch > 0) {
      const int per_b = p.Hkv * p.hchunks;
      const long long n_chunks = static_cast<long long>(p.ws_prefix[p.bsz]) * per_b;
      const long long at = before * per_b + static_cast<long long>(kvh * p.hchunks + hc) * nch;
      const int c0 = static_cast<int>(share_owner(at, n_chunks, n_own));
      const int c1 = static_cast<int>(share_owner(at + nch - 1, n_chunks, n_own));
      for (int k = (warp + W - taken % W) % W; k <= c1 - c0; k += W) {
        const float* src = k == 0
            ? p.ws_home + (static_cast<size_t>(b) * p.H + kvh * x.group + h) * dec::part_stride(D)
            : p.ws_cta + (static_cast<size_t>(c0 + k) * 8 + h % 8) * dec::part_stride(D);
        const float4 a = *reinterpret_cast<const float4*>(src + d0);
        const float4 c = *reinterpret_cast<const float4*>(src + d0 + 4);
        const float oc[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
        add(src[D], src[D + 1], oc);
      }
    }
  }
  sm[warp][lane] = m;
  sl[warp][lane] = l;
#pragma unroll
  for (int e = 0; e < 8; ++e) so[warp][e][lane] = o[e];
  __syncthreads();
  const int orow = threadIdx.x >> 3, e = threadIdx.x & 7;
  if (row0 + orow < x.rows) {
    float top = -INFINITY, sum = 0.f, acc = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmax3_nan(top, sm[w][orow], sm[w][orow]);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float mw = sm[w][orow];
      const float f = mw == -INFINITY ? 0.f : ex2_approx(mw - top);
      sum = fmaf(f, sl[w][orow], sum);
      acc = fmaf(f, so[w][e][orow], acc);
    }
    const int r = row0 + orow, b = r / x.group, h = r - b * x.group;
    out[(static_cast<size_t>(b) * x.H + kvh * x.group + h) * D + d0 + e] =
        __float2bfloat16_rn(sum == 0.f ? 0.f : acc / sum);
  }
}

}  // namespace la
