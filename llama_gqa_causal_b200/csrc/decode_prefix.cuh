// Decode for a batch whose sequences share a prefix: one query row per head
// against the prefix's rows and the sequence's own rows, in one softmax.
//
// For a K/V head the query rows of the whole batch (bsz x group of them) meet
// the same prefix, so that part is a product of matrices and runs on tcgen05:
//   S = Q K_prefix^T (128 query rows x 128 keys), P = 2^(S c - m), O += P V_prefix
// with each prefix tile read once for up to 256 query rows.  The sequences' own
// rows are a separate stream of 16-row tiles for mma.sync (own_share), as in
// the split-KV decode but with every warp a worker of its own.  Both parts run
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
//
// What bounds it: the prefix part's full tile pairs, like the prefill's tiles, the
// chain S -> softmax -> P -> P V -> S of either unit, which the other unit's half
// hides (a pair's 128 keys take 1.96 us an SM, 1.26 PFLOP/s over the chip, by what
// 128 sequences of 64/8 heads of 128 take more behind 65536 keys than behind
// 32768); shared tile pairs and the own rows, memory.  32 such sequences behind
// 8192 keys with 512 own rows on average (caches cold): 33 us for 102 MB; 128
// behind 32768: 142 us for 139 GFLOP.
// Few sequences with little behind them are taken whole by a block each
// (decode_prefix_small_kernel), which saves the second launch and the partials.
#pragma once
#include <type_traits>

#include "decode_bf16.cuh"

namespace la {
namespace px {
constexpr int BM = 128;      // query rows of a unit (= TMEM lanes)
constexpr int BN = 128;      // keys of a tile
constexpr int THREADS = 384;
constexpr int MAX_CTAS = 148;
// Ring of K and V tiles.  Five (what fits beside two Q tiles) streamed a prefix
// under 16 rows a head at 5.7 TB/s, four at 6.0; three took 2 us more for 32
// sequences behind 8192 keys.
__host__ __device__ constexpr int ring(int d) { return d == 128 ? 4 : 8; }
// The split of 384 x 168 registers: 56 + 224 + 224 a lane.
constexpr int kRegsControl = 56;
constexpr int kRegsSoftmax = 224;
constexpr int kRegsAtLaunch = (65536 / THREADS) / 8 * 8;  // 168
static_assert(kRegsControl % 8 == 0 && kRegsSoftmax % 8 == 0, "setmaxnreg takes multiples of 8");
static_assert(kRegsControl + 2 * kRegsSoftmax <= 3 * kRegsAtLaunch,
              "setmaxnreg split exceeds the registers the block is launched with");
constexpr float kRescaleThreshold = 8.0f;  // log2 units
// Pairs of 8 exponentiated on the FMA pipe instead of the MUFU: 0, 1 and 2 took
// 127, 123.5 and 123.5 us for 128 sequences behind 32768 keys.
constexpr int kPolyPairsOf8 = 1;
// What one SM takes, in microseconds as a mixed batch of 16 to 128 sequences ran
// (a prefix alone is a little sooner, 1.96 an item), for an item of a full and of a
// shared tile pair, a segment's beginning and end (Q, the pipeline's fill, the
// partial's write), and a step through the own rows.  Only their ratios matter.
__host__ __device__ constexpr float cost_pair(int d) { return d == 128 ? 2.1f : 1.5f; }
__host__ __device__ constexpr float cost_single(int d) { return d == 128 ? 1.6f : 1.1f; }
__host__ __device__ constexpr float cost_step(int d) { return d == 128 ? 0.12f : 0.07f; }
__host__ __device__ constexpr float cost_segment(int d) { return d == 128 ? 4.f : 2.f; }
// Floats of one unit's partial: [D + 2][BM], the outputs of a row down a
// column, then its maximum and sum (lanes are rows, so both the writing warp
// and the combining one touch whole lines).
__host__ __device__ constexpr int unit_floats(int d) { return (d + 2) * BM; }
// Own rows: warps of a CTA, stages of a warp, rows of a tile.
constexpr int OW = THREADS / 32;
__host__ __device__ constexpr int ow_min(int d) { return d == 128 ? 6 : 9; }
constexpr int OS = 2;
constexpr int OT = 16;
}  // namespace px

struct PrefixParams {
  const __nv_bfloat16* q;  // [b, H, D]
  float* part;             // prefix partials [tile pairs * Hkv + MAX_CTAS][2][D + 2][BM]
  float* own_home;         // [b * Hkv * hchunks][D + 2][heads]: from a sequence's first row
  float* own_mid;          // [MAX_CTAS * OW][D + 2][heads]: a worker's segment from inside one
  int2* part_of;           // [tile pairs * Hkv] CTA with the home slot, segments
  int2* own_of;            // [b * Hkv * hchunks] worker with the home slot, segments
  int rows;                // query rows of a K/V head: b * group
  int P;                   // keys of the prefix
  int nt;                  // its key tiles
  int pairs;               // tile pairs: ceil(rows / 256)
  int b, H, Hkv, L, group;
  int hchunks;             // ceil(group / 8)
  int heads;               // min(group, 8), the heads of a chunk's partial
  const int* lens;             // [b]
  const __nv_bfloat16* k_new;  // [b, Hkv, D] or null
  const __nv_bfloat16* v_new;
  __nv_bfloat16* k_cache;      // [b, Hkv, L, D]
  __nv_bfloat16* v_cache;
  float scale_log2;
};

// How many CTAs take a share of the prefix's items, and how many of the own rows.
struct PrefixPlan {
  int prefix, own;
};
__device__ __forceinline__ PrefixPlan prefix_plan(const PrefixParams& x, int n_steps, int n_ctas,
                                                  float c_pair, float c_single, float c_step,
                                                  float c_segment) {
  PrefixPlan r = {0, 0};
  const int runs = x.pairs * x.Hkv;  // of x.nt items
  if (x.nt > 0) {
    const bool single = x.rows - (x.pairs - 1) * 2 * px::BM <= px::BM;  // the last pair
    const float per_head = static_cast<float>(x.pairs - single) * c_pair + (single ? c_single : 0.f);
    const float wa = static_cast<float>(runs) * c_segment +
                     static_cast<float>(x.Hkv) * static_cast<float>(x.nt) * per_head;
    const float wb = static_cast<float>(n_steps) * c_step;
    // na with h + wa / na = wb / (n - na), where h is what a prefix CTA takes
    // besides its items and their segments (a split one among them) more than an
    // own one
    const float n = static_cast<float>(n_ctas), h = 2.f * c_segment;
    const float p = wa + wb - h * n, root = sqrtf(p * p + 4.f * h * wa * n);
    int na = n_ctas;
    if (n_steps > 0)  // (either form of the root, so that nothing cancels)
      na = static_cast<int>((p > 0.f ? 2.f * wa * n / (p + root) : (root - p) / (2.f * h)) + 0.5f);
    na = max(1, min(na, n_steps > 0 ? n_ctas - 1 : n_ctas));
    r.prefix = min(na, runs * x.nt);
    // whole CTAs to every run where that hands over few to the own rows (or idles
    // few): a CTA with one segment is done sooner than one that turns from one
    // run to the next (32 sequences behind 8192 keys 33.0 -> 31.3 us)
    const int over = r.prefix % runs;
    if (r.prefix > runs && over * 8 <= r.prefix) r.prefix -= over;
  }
  r.own = min(n_steps, n_ctas - r.prefix);
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
// for 2^f (largest relative error 7.5e-5, far below the 2^-8 that rounding the
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

// share_start in 32 bits: i n / g = i (n / g) + i (n % g) / g, for g^2 < 2^31.
__device__ __forceinline__ int share_begin(int i, int n, int g) {
  const int each = n / g;
  return i * each + i * (n - each * g) / g;
}

// A run of items inside one (tile pair, K/V head).
struct PrefixSegment {
  int seq, kvh;   // seq = tile pair * Hkv + kvh
  int row0, rows; // of the K/V head's query rows
  int j0, n;      // key tiles
  bool single;    // both units on the same rows, key tiles in turn
};
__device__ __forceinline__ PrefixSegment prefix_segment(const PrefixParams& x, int i0, int i1) {
  PrefixSegment g;
  g.seq = i0 / x.nt;
  g.j0 = i0 - g.seq * x.nt;
  g.n = min(x.nt - g.j0, i1 - i0);
  const int pair = g.seq / x.Hkv;
  g.kvh = g.seq - pair * x.Hkv;
  g.row0 = pair * 2 * px::BM;
  g.rows = min(2 * px::BM, x.rows - g.row0);
  g.single = g.rows <= px::BM;
  return g;
}

// One prefix CTA's run of items.
template <int D>
__device__ __forceinline__ void prefix_share(PrefixSmem<D>& s, const CUtensorMap& tm_k,
                                             const CUtensorMap& tm_v, const PrefixParams& x,
                                             int cta, int n_ctas) {
  using namespace px;
  constexpr int CB = D / 64;                  // 64-column swizzle blocks per row
  constexpr int NST = ring(D);
  constexpr uint32_t BLOCK_BYTES = BM * 128;  // one [128 rows x 64 cols] bf16 block
  constexpr uint32_t TILE_BYTES = BM * D * 2;
  constexpr uint32_t IDESC_QK = idesc_bf16(BM, BN, false);
  constexpr uint32_t IDESC_PV = idesc_bf16(BM, D, true);
  constexpr uint32_t TMEM_COLS = 512;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int items = x.pairs * x.Hkv * x.nt;
  const int x0 = share_begin(cta, items, n_ctas), x1 = share_begin(cta + 1, items, n_ctas);

  // ---- Q rows into a unit's tile, by its softmax warps: row m of the K/V head
  // is batch entry m / group, head kvh * group + m % group; a row's 16-byte
  // chunks go to adjacent lanes.  Rows past the end are zero.
  auto stage_q = [&](const PrefixSegment& g, int t) {
    constexpr int CH16 = D / 8;
    constexpr int RPS = 32 / CH16;
    const int r0 = (warp & 3) * 32 + lane / CH16, c = lane % CH16;
    const int rows = min(BM, g.rows - t * BM);
    // one division a call: the rows that follow are reached by adding
    const int m = g.row0 + t * BM + r0;
    const int b = m / x.group;
    int h = m - b * x.group;
    const __nv_bfloat16* src =
        x.q + (static_cast<size_t>(b) * x.H + g.kvh * x.group + h) * D + c * 8;
    const int h_step = RPS % x.group;
    const long long jump = static_cast<long long>(x.H - x.group) * D;  // to the next entry's heads
    const long long step = static_cast<long long>(RPS) * D + (RPS / x.group) * jump;
    uint4 v[32 / RPS];
#pragma unroll
    for (int st = 0; st < 32 / RPS; ++st) {
      v[st] = r0 + st * RPS < rows ? *reinterpret_cast<const uint4*>(src) : make_uint4(0, 0, 0, 0);
      src += step;
      h += h_step;
      if (h >= x.group) {
        h -= x.group;
        src += jump;
      }
    }
    uint8_t* qs = reinterpret_cast<uint8_t*>(&s.q[t][0]) + (c / 8) * BLOCK_BYTES;
#pragma unroll
    for (int st = 0; st < 32 / RPS; ++st)
      *reinterpret_cast<uint4*>(qs + sw128_offset(r0 + st * RPS, c % 8)) = v[st];
    fence_proxy_async_smem();
  };
  // ---- setup, with the first loads on their way: Q, and the first K tile (the
  // rest of the ring follows the sync, so that Q does not queue behind it)
  if (warp == 0) {
    if (elect_one()) {
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
      const PrefixSegment g = prefix_segment(x, x0, x1);
      mbar_arrive_expect_tx(&s.full[0], TILE_BYTES);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
        tma_load_3d(reinterpret_cast<uint8_t*>(&s.ring[0][0]) + cb * BLOCK_BYTES, &tm_k, &s.full[0],
                    cb * 64, g.j0 * BN, g.kvh);
    }
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(&s.tmem_base, TMEM_COLS);
    tmem_relinquish();
  } else if (warp >= 4) {
    const PrefixSegment g = prefix_segment(x, x0, x1);
    const int t = (warp - 4) >> 2;
    if (!g.single || t == 0) stage_q(g, t);
  }
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
    uint32_t sent = 1;  // tiles put into the ring
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
    for (int i = x0; i < x1 && ok;) {
      const PrefixSegment g = prefix_segment(x, i, x1);
      i += g.n;
      const int ahead = g.single ? 2 : 1;
      if (i > x0 + g.n) send(&tm_k, g.kvh, g.j0);  // (the very first is on its way)
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
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk / 4) * BLOCK_BYTES + (kk % 4) * 32) >> 4;
        mma_ss(tm_s(t), qd + off, kd + off, IDESC_QK, kk > 0 ? 1u : 0u);
      }
      tc_commit(&s.s_full[t]);
    };
    auto issue_pv = [&](int t, int st, bool accumulate, int h) {  // keys [64h, 64h + 64)
      const uint64_t vd = v_desc0 + ((static_cast<uint32_t>(st) * TILE_BYTES) >> 4);
#pragma unroll
      for (int kk = h * (BN / 32); kk < (h + 1) * (BN / 32); ++kk)
        mma_ts(tm_o(t), tm_s(t) + kk * 8, vd + ((kk * 2048) >> 4), IDESC_PV,
               (accumulate || kk > h * (BN / 32)) ? 1u : 0u);
    };
    // one lane does it all: it alone waits, so nothing lies between a barrier and
    // the products but their issue
    if (elect_one()) {
      // the ring: the next tile to be taken, and the parity of its full barrier
      int next_st = 0;
      uint32_t next_ph = 0;
      auto take = [&](int& st) {
        st = next_st;
        if (!mbar_wait(&s.full[st], next_ph)) return false;
        tc_fence_after();
        if (++next_st == NST) {
          next_st = 0;
          next_ph ^= 1;
        }
        return true;
      };
      uint32_t ph0 = 0, ph1 = 0;  // parity of each unit's next P tile
      uint32_t seg = 0;
      bool ok = true;
      for (int i = x0; i < x1 && ok; ++seg) {
        const PrefixSegment g = prefix_segment(x, i, x1);
        i += g.n;
        ok = mbar_wait(&s.q_ready[0], seg & 1) && mbar_wait(&s.q_ready[1], seg & 1);
        // step u of a segment is unit u & 1's, whether the units share the key
        // tiles (two steps a tile) or take them in turn; the code is laid out for
        // either unit, since what lies between a unit's P and the products is on
        // the path of every tile
        const int steps = g.single ? g.n : 2 * g.n;
        int vs = 0, ks = 0;
        auto step = [&](auto unit, int u) {
          constexpr int t = decltype(unit)::value;
          if (u >= 0) {  // O_t += P_t V
            if ((g.single || t == 0) && !take(vs)) return false;
            uint32_t& ph = t ? ph1 : ph0;
            if (!mbar_wait(&s.p_lo[t], ph)) return false;
            tc_fence_after();
            issue_pv(t, vs, u > 1, 0);
            if (!mbar_wait(&s.p_hi[t], ph)) return false;
            tc_fence_after();
            issue_pv(t, vs, true, 1);
            ph ^= 1;
            if (g.single || t == 1) tc_commit(&s.empty[vs]);
          }
          if (u + 2 < steps) {  // S_t = Q K^T of the unit's next tile
            if ((g.single || t == 0) && !take(ks)) return false;
            issue_qk(t, g.single ? 0 : t, ks);
            if (g.single || t == 1) tc_commit(&s.empty[ks]);
          } else {
            // (a unit without a tile waits for this all the same: running ahead, it
            // would complete two phases of q_ready between two of this warp's waits)
            tc_commit(&s.o_full[t]);
          }
          return true;
        };
#pragma unroll 1
        for (int u = -2; u < steps && ok; u += 2) {
          ok = step(std::integral_constant<int, 0>{}, u);
          if (ok && u + 1 < steps) ok = step(std::integral_constant<int, 1>{}, u + 1);
        }
      }
      // every MMA has completed before the CTA can exit
      tc_commit(&s.mma_done);
      mbar_wait(&s.mma_done, 0);
    }
    __syncwarp();
  } else if (warp < 4) {
    setmaxnreg_dec<kRegsControl>();
    // warp 2 notes where the combine kernel finds the segments of every (tile
    // pair, K/V head) that starts here; warp 3 brings the later segments' Q to L2
    if (warp == 3)
      for (int i = x0; i < x1;) {
        const PrefixSegment g = prefix_segment(x, i, x1);
        if (i > x0)
          for (int rr = lane; rr < g.rows; rr += 32) {
            const int m = g.row0 + rr;
            const int b = m / x.group, h = m - b * x.group;
            const __nv_bfloat16* row =
                x.q + (static_cast<size_t>(b) * x.H + g.kvh * x.group + h) * D;
            asm volatile("prefetch.global.L2 [%0];" ::"l"(row));
            if (D == 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 64));
          }
        i += g.n;
      }
    if (warp == 2 && lane == 0)
      for (int i = x0; i < x1;) {
        const PrefixSegment g = prefix_segment(x, i, x1);
        if (g.j0 == 0)
          x.part_of[g.seq] =
              make_int2(cta, static_cast<int>(share_owner(i + x.nt - 1, items, n_ctas)) - cta + 1);
        i += g.n;
      }
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
    if (lane == 0) mbar_arrive(&s.q_ready[t]);
#pragma unroll 1
    for (int i = x0; i < x1;) {
      const PrefixSegment g = prefix_segment(x, i, x1);
      i += g.n;
      const int rows = min(BM, g.rows - (g.single ? 0 : t) * BM);  // of this unit
      const bool active = quarter * 32 < rows;  // (warps past the rows only keep step)
      float m_ref = -INFINITY;  // reference maximum (log2 units) of the exponentials
      float l_sum = 0.f;
      const int n_mine = g.single ? (g.n + 1 - t) / 2 : g.n;
#pragma unroll 1
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
      // the next segment's Q first: its scores are taken while O is written out
      // (which no product touches before this unit's next P)
      if (i < x1) {
        const PrefixSegment next = prefix_segment(x, i, x1);
        if (!next.single || t == 0) stage_q(next, t);
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.q_ready[t]);
      }
      tc_fence_after();
      if (n_mine == 0) {  // (no tile: O is not this segment's)
        if (r < rows)
          for (int e = 0; e < D; ++e) dst[e * BM] = 0.f;
      } else if (active) {
#pragma unroll 1
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

// A warp's running softmax over 16-row tiles of keys for up to 8 query heads.
//   S^T[16 keys x 8 heads]  = K[16 x D] . Q^T[D x 8]
//   O^T[D x 8 heads]       += V^T[D x 16] . P^T[16 x 8]
// A lane holds the heads 2t, 2t + 1 (t = lane % 4); o[mt] has the dimensions
// mt * 16 + g and mt * 16 + g + 8 of either (g = lane / 4).
template <int D>
struct Tiles16 {
  static constexpr int KSTEPS = D / 16;
  static constexpr uint32_t BLOCK_BYTES = px::OT * 128;  // one [16 rows x 64 cols] block
  uint32_t qf[KSTEPS][2];
  float m[2], l[2], o[KSTEPS][4];

  // q: the first of n_heads heads
  __device__ __forceinline__ void start(const __nv_bfloat16* q, int n_heads) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const __nv_bfloat16* qr = q + g * D + 2 * t;  // dims kk * 16 + 2t + {0, 1, 8, 9}
#pragma unroll
    for (int kk = 0; kk < KSTEPS; ++kk) {
      qf[kk][0] = g < n_heads ? *reinterpret_cast<const uint32_t*>(qr + kk * 16) : 0u;
      qf[kk][1] = g < n_heads ? *reinterpret_cast<const uint32_t*>(qr + kk * 16 + 8) : 0u;
    }
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
#pragma unroll
    for (int mt = 0; mt < KSTEPS; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
  }

  // Rows from n_valid on may hold anything (V is zeroed there, so that a weight
  // of zero adds zero); patch: row n_valid - 1 is (kn, vn), a lane's 16 bytes.
  __device__ __forceinline__ void fix(uint8_t* kb, uint8_t* vb, int n_valid, bool patch,
                                      const uint4& kn, const uint4& vn) {
    const int lane = threadIdx.x & 31;
    constexpr int CB = D / 64;
    if (patch && lane < D / 8) {
      const uint32_t off = (lane / 8) * BLOCK_BYTES + sw128_offset(n_valid - 1, lane % 8);
      *reinterpret_cast<uint4*>(kb + off) = kn;
      *reinterpret_cast<uint4*>(vb + off) = vn;
    }
    for (int idx = lane; idx < (px::OT - n_valid) * CB * 8; idx += 32) {
      const int rr = n_valid + idx / (CB * 8), rem = idx % (CB * 8);
      *reinterpret_cast<uint4*>(vb + (rem / 8) * BLOCK_BYTES + sw128_offset(rr, rem % 8)) =
          make_uint4(0, 0, 0, 0);
    }
    if (patch || n_valid < px::OT) {
      fence_proxy_async_smem();  // (a copy may land here next)
      __syncwarp();
    }
  }

  __device__ __forceinline__ void add(const uint8_t* kb, const uint8_t* vb, int n_valid,
                                      float scale_log2) {
    const int lane = threadIdx.x & 31, g = lane >> 2;
    const int mat = lane >> 3, r8 = lane & 7;
    // ---- S^T = K Q^T, in two chains
    float sc[2][4] = {};
    const uint32_t kbase = smem_u32(kb), vbase = smem_u32(vb);
    const int krow = (mat & 1) * 8 + r8;
#pragma unroll
    for (int kk = 0; kk < KSTEPS; ++kk) {
      const int col = kk * 16 + (mat >> 1) * 8;
      uint32_t a0, a1, a2, a3;
      ldsm_x4(kbase + (col / 64) * BLOCK_BYTES + sw128_offset(krow, (col % 64) / 8), a0, a1, a2, a3);
      mma_bf16_16816(sc[kk & 1], a0, a1, a2, a3, qf[kk][0], qf[kk][1]);
    }
    // (key g, head 2t) (key g, head 2t + 1) (key g + 8, 2t) (key g + 8, 2t + 1)
    float pr[4], alpha[2];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      pr[e] = g + (e >> 1) * 8 < n_valid ? (sc[0][e] + sc[1][e]) * scale_log2 : -INFINITY;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(pr[h], pr[h + 2]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
      const float m_new = fmaxf(m[h], mx);
      const float ref = m_new == -INFINITY ? 0.f : m_new;
      alpha[h] = m[h] == -INFINITY ? 0.f : ex2_approx(m[h] - ref);
      pr[h] = ex2_approx(pr[h] - ref);
      pr[h + 2] = ex2_approx(pr[h + 2] - ref);
      l[h] = fmaf(l[h], alpha[h], pr[h] + pr[h + 2]);
      m[h] = m_new;
    }
#pragma unroll
    for (int mt = 0; mt < KSTEPS; ++mt) {
      o[mt][0] *= alpha[0];
      o[mt][1] *= alpha[1];
      o[mt][2] *= alpha[0];
      o[mt][3] *= alpha[1];
    }
    // P rounded to bf16 for the product; the sum is of the unrounded values
    const uint32_t pb0 = movmatrix_t(pack_bf16x2(pr[0], pr[1]));
    const uint32_t pb1 = movmatrix_t(pack_bf16x2(pr[2], pr[3]));
    // ---- O^T += V^T P^T
    const int vrow = (mat >> 1) * 8 + r8;
#pragma unroll
    for (int mt = 0; mt < KSTEPS; ++mt) {
      const int col = mt * 16 + (mat & 1) * 8;
      uint32_t a0, a1, a2, a3;
      ldsm_x4_t(vbase + (col / 64) * BLOCK_BYTES + sw128_offset(vrow, (col % 64) / 8), a0, a1, a2,
                a3);
      mma_bf16_16816(o[mt], a0, a1, a2, a3, pb0, pb1);
    }
  }

  // the sums over a head's keys (in every lane of the head)
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 4);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 8);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 16);
    }
  }
};

// The sequences' own rows.  A sequence here is (batch entry, K/V head, chunk of
// up to 8 query heads); its rows are cut into tiles of 16.  A sequence of n tiles
// counts n + 1 steps, the last of them empty: what starting and ending it takes
// (without it a warp with a share of one-tile sequences took half as long again
// as the others).  The steps of all sequences are numbered through, and every
// warp of every own CTA takes an even share of them.  A warp feeds itself (its
// own ring of tiles, one lane issuing the copies) and keeps its running softmax
// in registers, so no warp waits for another: with four warps of a block sharing
// 64-row tiles and merging at the end of every sequence, 1024 sequences of 256
// rows ran at 2.7 TB/s.
template <int D>
struct OwnSmem {
  alignas(1024) __nv_bfloat16 k[px::OW][px::OS][px::OT * D];
  alignas(1024) __nv_bfloat16 v[px::OW][px::OS][px::OT * D];
  uint64_t full[px::OW][px::OS];
  int before[dec::MAX_BATCH + 1];  // steps of one sequence each of the entries before b
};

// before[b] = steps of one sequence of each of the entries 0 .. b - 1, summed;
// every thread of the block takes part.
template <bool APPEND>
__device__ __forceinline__ void scan_steps(int* before, const PrefixParams& x) {
  using namespace px;
  auto steps = [&](int b) {
    const int len = attend_len(x.lens[b], x.L, APPEND);
    return len > 0 ? (len + OT - 1) / OT + 1 : 0;
  };
  __shared__ int warp_total[THREADS / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (x.b + THREADS - 1) / THREADS;
  const int lo = min(x.b, static_cast<int>(threadIdx.x) * per), hi = min(x.b, lo + per);
  int sum = 0;
  for (int b = lo; b < hi; ++b) sum += steps(b);
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  if (lane == 31) warp_total[warp] = incl;
  __syncthreads();
  int acc = incl - sum;
  for (int w = 0; w < warp; ++w) acc += warp_total[w];
  if (threadIdx.x == THREADS - 1) before[x.b] = acc + sum;
  for (int b = lo; b < hi; ++b) {
    before[b] = acc;
    acc += steps(b);
  }
  __syncthreads();
}

// A tile's place in the list of steps.
struct OwnCursor {
  int i;             // its step
  int b, seq, c, n;  // batch entry, sequence within it, tile of that, its tiles
};

template <int D, bool APPEND>
__device__ __forceinline__ void own_share(OwnSmem<D>& s, const CUtensorMap& tm_k,
                                          const CUtensorMap& tm_v, const PrefixParams& x,
                                          int worker, int n_workers, int n_steps) {
  using namespace px;
  constexpr int KSTEPS = D / 16;
  constexpr int CB = D / 64;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int per_b = x.Hkv * x.hchunks;
  const int x1 = share_begin(worker + 1, n_steps, n_workers);

  // to the next tile, over the empty step and the entries without a row
  auto advance = [&](OwnCursor& u) {
    ++u.i;
    if (++u.c < u.n) return;
    ++u.i;
    u.c = 0;
    if (++u.seq < per_b) return;
    u.seq = 0;
    do ++u.b;
    while (u.b < x.b && s.before[u.b + 1] == s.before[u.b]);
    u.n = u.b < x.b ? s.before[u.b + 1] - s.before[u.b] - 1 : 0;
  };
  OwnCursor at;  // of the tile in hand
  {
    at.i = share_begin(worker, n_steps, n_workers);
    int lo = 0, hi = x.b - 1;  // the largest b with before[b] * per_b <= at.i
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (s.before[mid] * per_b <= at.i) lo = mid;
      else hi = mid - 1;
    }
    const int steps = s.before[lo + 1] - s.before[lo];
    const int rest = at.i - s.before[lo] * per_b;
    at.b = lo;
    at.n = steps - 1;
    at.seq = rest / steps;
    at.c = rest - at.seq * steps;
    if (at.c == at.n) {  // the share starts at an empty step
      --at.i;
      --at.c;
      advance(at);
    }
  }
  OwnCursor to = at;  // of the next tile to be fetched
  int fetched = 0;
  // the tile at `to`; with a sequence's first tile its query rows, with its last
  // one the step's own row are brought to L2, so that a share of many short
  // sequences does not pay for each from memory
  auto fetch = [&]() {
    const int st = fetched % OS;
    const int kvh = to.seq / x.hchunks, hc = to.seq - kvh * x.hchunks;
    const int bh = to.b * x.Hkv + kvh;
    if (to.c == 0 && fetched > 0 && lane < 8 * CB && hc * 8 + lane / CB < x.group)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          x.q + (static_cast<size_t>(to.b) * x.H + kvh * x.group + hc * 8 + lane / CB) * D +
          lane % CB * 64));
    if (APPEND && to.c + 1 == to.n && lane < 2 * CB)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(
          (lane < CB ? x.k_new : x.v_new) + static_cast<size_t>(bh) * D + lane % CB * 64));
    if (elect_one()) {
      mbar_arrive_expect_tx(&s.full[warp][st], 2u * OT * D * 2u);
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        tma_load_3d(&s.k[warp][st][cb * OT * 64], &tm_k, &s.full[warp][st], cb * 64, to.c * OT, bh);
        tma_load_3d(&s.v[warp][st][cb * OT * 64], &tm_v, &s.full[warp][st], cb * 64, to.c * OT, bh);
      }
    }
    __syncwarp();
    ++fetched;
    advance(to);
  };
#pragma unroll 1
  for (int k = 0; k < OS && to.i < x1; ++k) fetch();

  Tiles16<D> st16;
  bool home = false;
  int len = 0;
  for (int k = 0; at.i < x1; ++k) {
    const int st = k % OS;
    const int kvh = at.seq / x.hchunks, hc = at.seq - kvh * x.hchunks;
    if (k == 0 || at.c == 0) {  // a segment starts
      home = at.c == 0;
      if (home) {
        const int n = at.i + at.n <= x1 ? 1
            : static_cast<int>(share_owner(at.i + at.n - 1, n_steps, n_workers)) - worker + 1;
        if (lane == 0) x.own_of[at.b * per_b + at.seq] = make_int2(worker, n);
      }
      len = attend_len(x.lens[at.b], x.L, APPEND);
      st16.start(x.q + (static_cast<size_t>(at.b) * x.H + kvh * x.group + hc * 8) * D,
                 x.group - hc * 8);
    }
    const int n_valid = min(OT, len - at.c * OT);
    const bool patch = APPEND && at.c == at.n - 1;  // the step's own row is the last
    const size_t bh = static_cast<size_t>(at.b) * x.Hkv + kvh;
    uint4 kn, vn;
    if (patch && lane < D / 8) {  // (on their way while the tile is waited for)
      kn = *reinterpret_cast<const uint4*>(x.k_new + bh * D + lane * 8);
      vn = *reinterpret_cast<const uint4*>(x.v_new + bh * D + lane * 8);
    }
    if (!mbar_wait(&s.full[warp][st], static_cast<uint32_t>(k / OS) & 1)) {
      // (given up: the status word is set; leave no copy in flight)
      for (int j = k; j < fetched; ++j)
        mbar_wait(&s.full[warp][j % OS], static_cast<uint32_t>(j / OS) & 1);
      return;
    }
    uint8_t* kb = reinterpret_cast<uint8_t*>(&s.k[warp][st][0]);
    uint8_t* vb = reinterpret_cast<uint8_t*>(&s.v[warp][st][0]);
    if (patch && hc == 0 && lane < D / 8) {
      const size_t crow = (bh * x.L + (len - 1)) * D + lane * 8;
      *reinterpret_cast<uint4*>(x.k_cache + crow) = kn;
      *reinterpret_cast<uint4*>(x.v_cache + crow) = vn;
    }
    st16.fix(kb, vb, n_valid, patch, kn, vn);
    st16.add(kb, vb, n_valid, x.scale_log2);
    __syncwarp();
    if (to.i < x1) fetch();
    if (at.i + 1 >= x1 || at.c + 1 == at.n) {  // the segment ends: its partial
      st16.finish();
      float* dst = (home ? x.own_home + static_cast<size_t>(at.b * per_b + at.seq) * (D + 2) * x.heads
                         : x.own_mid + static_cast<size_t>(worker) * (D + 2) * x.heads) +
                   2 * t;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (hc * 8 + 2 * t + h < x.group) {
#pragma unroll
          for (int mt = 0; mt < KSTEPS; ++mt) {
            dst[(mt * 16 + g) * x.heads + h] = st16.o[mt][h];
            dst[(mt * 16 + g + 8) * x.heads + h] = st16.o[mt][h + 2];
          }
          if (g == 0) {
            dst[D * x.heads + h] = st16.m[h];
            dst[(D + 1) * x.heads + h] = st16.l[h];
          }
        }
      }
    }
    advance(at);
  }
}

template <int D>
constexpr size_t prefix_smem_bytes() {
  return (sizeof(PrefixSmem<D>) > sizeof(OwnSmem<D>) ? sizeof(PrefixSmem<D>) : sizeof(OwnSmem<D>)) +
         1024;
}

template <int D, bool APPEND>
__global__ void __launch_bounds__(px::THREADS, 1)
    decode_prefix_kernel(const __grid_constant__ CUtensorMap tm_kp,
                         const __grid_constant__ CUtensorMap tm_vp,
                         const __grid_constant__ CUtensorMap tm_k,
                         const __grid_constant__ CUtensorMap tm_v,
                         const __grid_constant__ PrefixParams x) {
  using namespace px;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  OwnSmem<D>& own = *reinterpret_cast<OwnSmem<D>*>(smem);
  // a programmatic dependent of what precedes it: no global memory before this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  {
    // q to L2 while the lengths are read: where its rows go is only known then
    const size_t line = static_cast<size_t>(blockIdx.x) * THREADS + threadIdx.x;
    if (line < static_cast<size_t>(x.b) * x.H * D / 64)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(x.q + line * 64));
  }
  scan_steps<APPEND>(own.before, x);
  const int n_steps = own.before[x.b] * x.Hkv * x.hchunks;
  const PrefixPlan plan =
      prefix_plan(x, n_steps, gridDim.x, cost_pair(D), cost_single(D), cost_step(D),
                  cost_segment(D));
  // warps of an own CTA: all 12, or as many as make ow_min a CTA of the whole
  // chip.  Reads under way from more places than that make memory slower: 32
  // sequences of 4096 own rows, 146 own CTAs, 117 us with 12 warps, 90 with 6
  // (heads of 64, half the bytes a tile: 59 with 12, 55 with 8, 68 with 6); with
  // 68 own CTAs beside the prefix's, 8 warps were 6% slower than 12.
  const int own_warps =
      plan.own > 0 ? min(OW, max(ow_min(D), ow_min(D) * MAX_CTAS / plan.own)) : OW;
  const int n_workers = min(n_steps, plan.own * own_warps);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // own CTAs evenly among the others, so that no part of the chip has only the
  // ones or the others on its way to memory
  const int n = gridDim.x;
  const int own_before = blockIdx.x * plan.own / n;
  if ((blockIdx.x + 1) * plan.own / n == own_before) {
    const int cta = blockIdx.x - own_before;
    if (cta >= plan.prefix) return;
    // the scan's shared memory has been read, and the ring's copies may land there
    fence_proxy_async_smem();
    __syncthreads();
    prefix_share<D>(*reinterpret_cast<PrefixSmem<D>*>(smem), tm_kp, tm_vp, x, cta, plan.prefix);
    return;
  }
  // warps of one CTA are workers plan.own apart, so that few tiles spread over the SMs
  const int worker = own_before + (threadIdx.x >> 5) * plan.own;
  if (worker >= n_workers) return;
  if ((threadIdx.x & 31) == 0) {
    for (int i = 0; i < OS; ++i) mbar_init(&own.full[threadIdx.x >> 5][i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  own_share<D, APPEND>(own, tm_k, tm_v, x, worker, n_workers, n_steps);
}

// Merges the partials of 32 query rows of one K/V head: a lane is a row, a warp
// 8 of its dimensions, and WK warps with the same dimensions take the partials
// in turn and are merged through shared memory.  Bound by the latency of its
// loads: U = 2 partials at a time in 64 registers, which lets four blocks into an
// SM, was faster than U = 4 with three (35.0 against 36.3 us for 32 sequences behind
// 8192 tokens).
namespace px {
constexpr int COMBINE_WARPS = 8;
}
template <int D, int WK>
__global__ void __launch_bounds__(px::COMBINE_WARPS * 32, 4)
    decode_prefix_combine_kernel(const __grid_constant__ PrefixParams x, int append,
                                 __nv_bfloat16* __restrict__ out) {
  using namespace px;
  constexpr int WD = COMBINE_WARPS / WK;  // warps side by side over the dimensions
  constexpr int DC = D / (8 * WD);        // blocks over the dimensions
  constexpr int U = 2;  // partials loaded at a time
  __shared__ float so[COMBINE_WARPS][10][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int wk = warp / WD, wd = warp - wk * WD;
  const int rb = static_cast<int>(blockIdx.x / DC);
  const int d0 = (static_cast<int>(blockIdx.x - rb * DC) * WD + wd) * 8;
  const int blocks_per_kvh = (x.rows + 31) / 32;
  const int kvh = rb / blocks_per_kvh;
  const int row0 = (rb - kvh * blocks_per_kvh) * 32;
  const bool valid = row0 + lane < x.rows;
  const int row = min(row0 + lane, x.rows - 1);
  const int b = row / x.group, h = row - b * x.group;
  const int pair = row0 / (2 * BM), in_pair = row0 - pair * 2 * BM;
  const bool single = x.rows - pair * 2 * BM <= BM;
  const int seq = pair * x.Hkv + kvh;
  const int own_seq = (b * x.Hkv + kvh) * x.hchunks + h / 8;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int2 pre = x.nt > 0 ? x.part_of[seq] : make_int2(0, 0);
  int2 own = x.own_of[own_seq];
  if (attend_len(x.lens[b], x.L, append) == 0) own = make_int2(0, 0);  // (nothing was noted)

  float m = -INFINITY, l = 0.f, o[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
  // merges U partials; one that is not there has the maximum -inf and zeros
  auto add = [&](const float (&mc)[U], const float (&lc)[U], const float (&oc)[U][8]) {
    float top = m;
#pragma unroll
    for (int u = 0; u < U; ++u) top = fmax3_nan(top, mc[u], mc[u]);
    const float ref = top == -INFINITY ? 0.f : top;
    const float f = ex2_approx(m - ref);
    l *= f;
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] *= f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float w = ex2_approx(mc[u] - ref);
      l = fmaf(w, lc[u], l);
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(w, oc[u][e], o[e]);
    }
    m = top;
  };
  // the partials: of the prefix the home slot, then those of the CTAs that follow
  // its CTA, two units each if they share their rows; of the own rows the home
  // slot, then those of the workers that follow.  A column of each holds one row.
  const int n_pre = pre.y << single, n = n_pre + own.y;
  const float* base = x.part + in_pair / BM * unit_floats(D) + in_pair % BM + lane;
  for (int k0 = wk; k0 < n; k0 += U * WK) {
    float mc[U], lc[U], oc[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = k0 + u * WK;
      const float* src;
      int stride = BM;
      if (k < n_pre) {
        const int seg = k >> single;
        const int slot = seg == 0 ? seq : x.pairs * x.Hkv + pre.x + seg;
        src = base + static_cast<long long>(2 * slot + (single ? k & 1 : 0)) * unit_floats(D);
      } else {
        const int seg = k - n_pre;
        const long long slot = seg == 0 ? own_seq : own.x + seg;
        stride = x.heads;
        src = (seg == 0 ? x.own_home : x.own_mid) + slot * (D + 2) * stride + h % 8;
      }
      const bool there = valid && k < n;
      mc[u] = there ? src[D * stride] : -INFINITY;
      lc[u] = there ? src[(D + 1) * stride] : 0.f;
      src += d0 * stride;
#pragma unroll
      for (int e = 0; e < 8; ++e) oc[u][e] = there ? src[e * stride] : 0.f;
    }
    add(mc, lc, oc);
  }
  so[warp][8][lane] = m;
  so[warp][9][lane] = l;
#pragma unroll
  for (int e = 0; e < 8; ++e) so[warp][e][lane] = o[e];
  __syncthreads();
  // a warp takes 8 / WK of its dimensions over all WK warps that have them
  constexpr int E = 8 / WK;
  const int e0 = wk * E;
  float top = -INFINITY, sum = 0.f, acc[E];
#pragma unroll
  for (int w = 0; w < WK; ++w) {
    const float mw = so[w * WD + wd][8][lane];
    top = fmax3_nan(top, mw, mw);
  }
  const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll
  for (int w = 0; w < WK; ++w) {
    const float f = ex2_approx(so[w * WD + wd][8][lane] - ref);
    sum = fmaf(f, so[w * WD + wd][9][lane], sum);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(f, so[w * WD + wd][e0 + e][lane], acc[e]);
  }
  if (!valid) return;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat16* dst = out + (static_cast<size_t>(b) * x.H + kvh * x.group + h) * D + d0 + e0;
  if constexpr (E == 1) {
    *dst = __float2bfloat16_rn(acc[0] * inv);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  }
}

// Sequences with little behind them: a block takes one sequence (batch entry, K/V
// head, chunk of up to 8 query heads) from beginning to end, its W warps the
// 16-row tiles of prefix and own rows in turn, each through a ring of its own,
// and merges them through shared memory.  One launch and no partials, but each
// block reads the prefix for itself (out of L2, mostly) and a long one makes it
// late.  The warps read rows that lie next to one another, and 144 sequences of
// 4000 own rows run at 6.5 TB/s.  16 sequences x 8 K/V heads behind 500 + 100
// rows: 6.1 us, against 14.9 split over the SMs; behind 3000 + 100: 17.4, 17.8.
// W = 8 where a wave of such blocks (166 KB of shared memory, 81 KB for heads of
// 64) holds all sequences, else 4, of which two (five) fit an SM: 1024 sequences
// behind 20 rows 10.8 us against 18.3, but 144 behind 1000 12.6 against 9.4.
template <int D, int W>
struct SmallSmem {
  alignas(1024) __nv_bfloat16 k[W][px::OS][px::OT * D];
  alignas(1024) __nv_bfloat16 v[W][px::OS][px::OT * D];
  float o[W][8][D + 4];  // (+ 4 spreads the rows over the banks)
  float m[W][8], l[W][8];
  uint64_t full[W][px::OS];
};
template <int D, bool APPEND, int W>
__global__ void __launch_bounds__(W * 32)
    decode_prefix_small_kernel(const __grid_constant__ CUtensorMap tm_kp,
                               const __grid_constant__ CUtensorMap tm_vp,
                               const __grid_constant__ CUtensorMap tm_k,
                               const __grid_constant__ CUtensorMap tm_v,
                               const __grid_constant__ PrefixParams x,
                               __nv_bfloat16* __restrict__ out) {
  using namespace px;
  constexpr int CB = D / 64;
  extern __shared__ uint8_t smem_raw[];
  SmallSmem<D, W>& s = *reinterpret_cast<SmallSmem<D, W>*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per_b = x.Hkv * x.hchunks;
  const int b = blockIdx.x / per_b, seq = blockIdx.x - b * per_b;
  const int kvh = seq / x.hchunks, hc = seq - kvh * x.hchunks;
  const int bh = b * x.Hkv + kvh;
  const int n_heads = min(8, x.group - hc * 8);
  const size_t row0 = static_cast<size_t>(b) * x.H + kvh * x.group + hc * 8;  // of q and out
  if (lane == 0) {
    for (int i = 0; i < OS; ++i) mbar_init(&s.full[warp][i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int n_pre = (x.P + OT - 1) / OT;
  auto fetch = [&](int i, int st) {  // tile i: of the prefix first, then the own rows
    if (elect_one()) {
      mbar_arrive_expect_tx(&s.full[warp][st], 2u * OT * D * 2u);
      const bool pre = i < n_pre;
      const CUtensorMap* mk = pre ? &tm_kp : &tm_k;
      const CUtensorMap* mv = pre ? &tm_vp : &tm_v;
      const int row = (pre ? i : i - n_pre) * OT, head = pre ? kvh : bh;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        tma_load_3d(&s.k[warp][st][cb * OT * 64], mk, &s.full[warp][st], cb * 64, row, head);
        tma_load_3d(&s.v[warp][st][cb * OT * 64], mv, &s.full[warp][st], cb * 64, row, head);
      }
    }
    __syncwarp();
  };
  // the prefix's length is known, the own rows' still has to be read
  int fetched = 0;
  for (; fetched < OS && warp + fetched * W < n_pre; ++fetched) fetch(warp + fetched * W, fetched);
  Tiles16<D> t16;
  t16.start(x.q + row0 * D, n_heads);
  const int len = attend_len(x.lens[b], x.L, APPEND);
  const int n = n_pre + (len + OT - 1) / OT;
  for (; fetched < OS && warp + fetched * W < n; ++fetched) fetch(warp + fetched * W, fetched);
  uint4 kn = make_uint4(0, 0, 0, 0), vn = kn;
  const bool mine = APPEND && (n - 1) % W == warp && lane < D / 8;  // the step's own row
  if (mine) {
    kn = *reinterpret_cast<const uint4*>(x.k_new + static_cast<size_t>(bh) * D + lane * 8);
    vn = *reinterpret_cast<const uint4*>(x.v_new + static_cast<size_t>(bh) * D + lane * 8);
  }
  bool ok = true;
  for (int i = warp, k = 0; i < n; i += W, ++k) {
    const int st = k % OS;
    if (!mbar_wait(&s.full[warp][st], static_cast<uint32_t>(k / OS) & 1)) {
      for (int j = k; j < fetched; ++j)  // (given up: leave no copy in flight)
        mbar_wait(&s.full[warp][j % OS], static_cast<uint32_t>(j / OS) & 1);
      ok = false;
      break;
    }
    uint8_t* kb = reinterpret_cast<uint8_t*>(&s.k[warp][st][0]);
    uint8_t* vb = reinterpret_cast<uint8_t*>(&s.v[warp][st][0]);
    const int n_valid = min(OT, i < n_pre ? x.P - i * OT : len - (i - n_pre) * OT);
    t16.fix(kb, vb, n_valid, APPEND && i == n - 1, kn, vn);
    t16.add(kb, vb, n_valid, x.scale_log2);
    __syncwarp();
    if (i + OS * W < n) {
      fetch(i + OS * W, st);
      ++fetched;
    }
  }
  if (mine && hc == 0 && ok) {
    const size_t crow = (static_cast<size_t>(bh) * x.L + (len - 1)) * D + lane * 8;
    *reinterpret_cast<uint4*>(x.k_cache + crow) = kn;
    *reinterpret_cast<uint4*>(x.v_cache + crow) = vn;
  }
  t16.finish();
  const int g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float* dst = s.o[warp][2 * t + h];
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt) {
      dst[mt * 16 + g] = t16.o[mt][h];
      dst[mt * 16 + g + 8] = t16.o[mt][h + 2];
    }
    if (g == 0) {
      s.m[warp][2 * t + h] = t16.m[h];
      s.l[warp][2 * t + h] = t16.l[h];
    }
  }
  __syncthreads();
  constexpr int VEC = D / 32;
  for (int hd = warp; hd < n_heads; hd += W) {
    float top = -INFINITY, sum = 0.f, acc[VEC];
#pragma unroll
    for (int w = 0; w < W; ++w) top = fmax3_nan(top, s.m[w][hd], s.m[w][hd]);
    const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
    for (int e = 0; e < VEC; ++e) acc[e] = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float f = ex2_approx(s.m[w][hd] - ref);
      sum = fmaf(f, s.l[w][hd], sum);
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = fmaf(f, s.o[w][hd][lane * VEC + e], acc[e]);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    __nv_bfloat16* dst = out + (row0 + hd) * D + lane * VEC;
#pragma unroll
    for (int e = 0; e < VEC; e += 2)
      *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(acc[e] * inv, acc[e + 1] * inv);
  }
}

}  // namespace la
