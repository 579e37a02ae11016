// Attention weight that each key receives from a set of queries: with the
// scores s of fa_score.cuh and the forward's log-sums,
//     w_j = sum over the kv head's query heads h and the queries i that may
//           see j of  e^(s_hij - lse_hi).
// It is the first half of the backward (scores recomputed, no row reduction
// needed) followed by a sum along queries, so the tile is taken transposed:
// S^T = K Q^T puts one key per TMEM lane, and each thread adds up its own key's
// probabilities in a register.  No score leaves the SM.
//
// Floor: 2 D FLOP and one exponential per pair.  The MUFU unit (16 exponentials
// per clock and SM, 1024 cycles for a 128 x 128 tile) bounds it before the
// tensor core does (512 cycles at D = 128).  Measured: a causal prompt of 4095
// tokens, 32 query and 8 kv heads of D = 128, 101 us (its exponentials alone:
// 58 us; the MUFU unit is 71% busy while an SM has work); the last 64 queries of
// 4 prompts over 8192 keys with a cap, 58 us (an item then holds four pairs of
// half-empty tiles, and what a pair costs besides its exponentials counts).
// Four neighbouring key tiles per item, one per warpgroup, so that no sums are
// joined and a Q tile is read once for the four, measured 120 and 73 us: the
// causal edge leaves warpgroups idle, and one product thread feeds four tiles a
// pair.
//
// The grid is persistent (one CTA per SM).  A work item is one (batch, kv head,
// 128-key tile, part); the (query tile, head of the group) pairs of the first
// three are dealt to `parts` items when there are too few of them for the SMs,
// and kw_reduce_kernel then adds the parts in a fixed order (no atomics: the
// result does not depend on timing).
//   warp 16     TMA: K of the item (two buffers), Q pair by pair (NQ stages)
//   warp 17     tcgen05: S^T of each pair into one of four TMEM buffers
//   warps 18, 19  -LSE in log2 units of every other pair's queries to shared
//               memory, the next pair's on its way meanwhile
//   warps 0-15  four warpgroups that take the pairs in turn, one thread per key,
//               by a rolled loop over 32 queries, or 16 with a cap, whose code is
//               longer (two warpgroups leave the sub-partitions idle on TMEM
//               loads and dependences: 147 against 126 us for the prompt above)
//   warp 17     also allocates TMEM
#pragma once
#include "sm100.cuh"
#include "fa_score.cuh"

namespace fa {

// n / d for 0 <= n < 2^31 by one wide product: floor(n m / 2^(31 + l)) with
// l = ceil(log2 d) and m = ceil(2^(31 + l) / d) < 2^32 is exact there, since m d
// exceeds 2^(31 + l) by less than d <= 2^l.
struct FastDiv {
  uint32_t d, m, s;
  __host__ static FastDiv of(uint32_t d) {
    uint32_t l = 0;
    while ((1u << l) < d) ++l;
    return {d, static_cast<uint32_t>(((uint64_t(1) << (31 + l)) + d - 1) / d), 31 + l};
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * m) >> s);
  }
  __device__ __forceinline__ int divmod(int n, int& rem) const {
    const int q = div(n);
    rem = n - q * static_cast<int>(d);
    return q;
  }
};

struct KwParams {
  const float* lse;      // [B, Hq, Lq]
  float* out;            // [B, Hkv, ld] (parts == 1) or the partial sums [parts, B, Hkv, ceil(Lk / 128) * 128]
  int ld, accumulate;    // parts == 1: row length of out, add to it or overwrite
  int B, Hq, Hkv, Lq, Lk, parts, num_items;
  FastDiv by_tile, by_parts, by_hkv, by_group;   // B Hkv parts; parts; Hkv; Hq / Hkv
  float scale_log2;
  uint64_t wait_limit_ns;
  ScoreParams sc;
};

template <int D>
struct KwCfg {
  static constexpr int TILE = 128 * D * 2;
  static constexpr int NQ = 4;                        // Q stages
  static constexpr int NS = 4;                        // S^T buffers in TMEM (4 x 128 columns)
  static constexpr int NR = 4;                        // LSE rows in shared memory
  static constexpr int K_OFF = 0;                     // two K buffers
  static constexpr int Q_OFF = 2 * TILE;
  static constexpr int ROW_OFF = Q_OFF + NQ * TILE;   // NR x 128 floats
  static constexpr int SUM_OFF = ROW_OFF + NR * 512;  // 3 x 128 floats: the other warpgroups' sums
  static constexpr int BAR_OFF = SUM_OFF + 3 * 512;
  static constexpr int NBARS = 4 + 2 * NQ + 2 * NS + 2 * NR + 2 + 1;
  static constexpr int SMEM_BYTES = BAR_OFF + NBARS * 8 + 16 + 1024;
  static constexpr int THREADS = 640;
};

enum : uint32_t {
  W_KW_K = 0x501, W_KW_K_FREE = 0x502, W_KW_Q = 0x503, W_KW_Q_EMPTY = 0x504, W_KW_S = 0x505, W_KW_S_FREE = 0x506,
  W_KW_ROW = 0x507, W_KW_ROW_EMPTY = 0x508, W_KW_SUM = 0x509, W_KW_SUM_FREE = 0x50a, W_KW_DONE = 0x50b,
  W_KW_DRAIN = 0x50c, W_IDX_KW_OUT = 0x408
};

struct KwItem {
  int b, hkv, j, part, i0, n0, n1;   // pairs [n0, n1): query tile i0 + n / G, head n % G
  int kuni, pre;
};
// Items are numbered key tile by key tile: under the causal mask the first ones
// are the heaviest.  CTA c takes, in round rd, item rd * G + c (rd even) or
// rd * G + G - 1 - c (rd odd) of G CTAs, which evens that out; j < 0: none.
__device__ __forceinline__ KwItem kw_item(const KwParams& p, int rd) {
  KwItem I;
  const int grid = static_cast<int>(gridDim.x), c = static_cast<int>(blockIdx.x);
  const int w = rd * grid + ((rd & 1) ? grid - 1 - c : c);
  I.j = -1;
  I.n0 = I.n1 = 0;
  if (w >= p.num_items) return I;
  const ScoreParams& sc = p.sc;
  const int nk = (p.Lk + 127) >> 7, nq = (p.Lq + 127) >> 7, G = p.Hq / p.Hkv;
  int rest;
  I.j = p.by_tile.divmod(w, rest);
  rest = p.by_parts.divmod(rest, I.part);
  I.b = p.by_hkv.divmod(rest, I.hkv);
  I.pre = sc.causal ? score_prefix(sc, I.b, p.Lk) : 0;
  I.i0 = 0;
  int i1 = nq;
  if (sc.causal && I.j * 128 >= I.pre) {
    const int first_q = I.j * 128 - (p.Lk - p.Lq);
    I.i0 = first_q <= 0 ? 0 : first_q >> 7;
  }
  I.kuni = -1;
  if (sc.q_docs != nullptr) {
    const int4 m = sc.k_meta[static_cast<size_t>(I.b) * nk + I.j];
    I.kuni = m.x;
    I.i0 = max(I.i0, m.y);
    i1 = min(i1, m.z);
  }
  const int n = max(0, i1 - I.i0) * G;             // n * 64 < 2^31
  I.n0 = p.by_parts.div(n * I.part);
  I.n1 = p.by_parts.div(n * (I.part + 1));
  return I;
}

template <int D, int MOD>
__global__ void __launch_bounds__(640, 1)
kw_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k, const KwParams p) {
  using C = KwCfg<D>;
  constexpr int NQ = C::NQ, NS = C::NS, NR = C::NR, KB = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);   // [2]
  uint64_t* k_free = k_full + 2;                                       // [2]
  uint64_t* q_full = k_free + 2;
  uint64_t* q_empty = q_full + NQ;
  uint64_t* s_full = q_empty + NQ;
  uint64_t* s_free = s_full + NS;
  uint64_t* r_full = s_free + NS;
  uint64_t* r_empty = r_full + NR;
  uint64_t* sum_full = r_empty + NR;
  uint64_t* sum_free = sum_full + 1;
  uint64_t* mma_done = sum_free + 1;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = p.wait_limit_ns;
  const int G = p.Hq / p.Hkv, off = p.Lk - p.Lq;

  if (threadIdx.x == 0) {
    for (int u = 0; u < 2; ++u) { mbar_init(&k_full[u], 1); mbar_init(&k_free[u], 1); }
    for (int u = 0; u < NQ; ++u) { mbar_init(&q_full[u], 1); mbar_init(&q_empty[u], 1); }
    for (int u = 0; u < NS; ++u) { mbar_init(&s_full[u], 1); mbar_init(&s_free[u], 128); }
    for (int u = 0; u < NR; ++u) { mbar_init(&r_full[u], 1); mbar_init(&r_empty[u], 128); }
    mbar_init(sum_full, 384);
    mbar_init(sum_free, 128);
    mbar_init(mma_done, 1);
    fence_mbar_init();
  }
  if (warp == 17) { tmem_alloc(tmem_holder, 512); tmem_relinquish(); }
  if (warp == 16 && lane == 0) { tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_k); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  pdl_wait();                                      // the tile facts of the documents

  if (warp == 16) {
    // ------------------------------------------------------------ producer --
    if (lane == 0) {
      int it = 0, gp = 0;                          // items with pairs, pairs issued
      bool ok = true;
      for (int rd = 0; ok && rd * static_cast<int>(gridDim.x) < p.num_items; ++rd) {
        const KwItem I = kw_item(p, rd);
        if (I.n0 == I.n1) continue;
        const int u = it & 1;
        if (it >= 2 && !(ok = mbar_wait(&k_free[u], ((it >> 1) + 1) & 1, lim, W_KW_K_FREE))) break;
        mbar_arrive_expect_tx(&k_full[u], C::TILE);
        for (int kb = 0; kb < KB; ++kb)
          tma_load_4d(smem + C::K_OFF + u * C::TILE + kb * 16384, &tm_k, &k_full[u], kb * 64, I.hkv, I.j * 128, I.b);
        ++it;
        for (int n = I.n0; n < I.n1; ++n, ++gp) {
          const int s = gp % NQ;
          int h;
          const int i = p.by_group.divmod(n, h);
          if (gp >= NQ && !(ok = mbar_wait(&q_empty[s], ((gp / NQ) + 1) & 1, lim, W_KW_Q_EMPTY))) break;
          mbar_arrive_expect_tx(&q_full[s], C::TILE);
          for (int kb = 0; kb < KB; ++kb)
            tma_load_4d(smem + C::Q_OFF + s * C::TILE + kb * 16384, &tm_q, &q_full[s], kb * 64, I.hkv * G + h,
                        (I.i0 + i) * 128, I.b);
        }
      }
      // the CTA may not exit with copies in flight
      for (int k = max(0, it - 2); k < it; ++k) mbar_wait(&k_full[k & 1], (k >> 1) & 1, lim, W_KW_DRAIN);
      for (int g = max(0, gp - NQ); g < gp; ++g) mbar_wait(&q_full[g % NQ], (g / NQ) & 1, lim, W_KW_DRAIN);
    }
  } else if (warp == 17) {
    // ----------------------------------------------------------------- MMA --
    if (lane == 0) {
      constexpr uint32_t IDESC = idesc_bf16_f32(128, 128, false, false);
      const uint32_t kb0 = smem_u32(smem + C::K_OFF), qb0 = smem_u32(smem + C::Q_OFF);
      int it = 0, gp = 0;
      bool ok = true;
      for (int rd = 0; ok && rd * static_cast<int>(gridDim.x) < p.num_items; ++rd) {
        const KwItem I = kw_item(p, rd);
        if (I.n0 == I.n1) continue;
        const int u = it & 1;
        if (!(ok = mbar_wait(&k_full[u], (it >> 1) & 1, lim, W_KW_K))) break;
        for (int n = I.n0; n < I.n1; ++n, ++gp) {
          const int s = gp % NQ, t = gp % NS;
          if (!(ok = mbar_wait(&q_full[s], (gp / NQ) & 1, lim, W_KW_Q))) break;
          if (gp >= NS && !(ok = mbar_wait(&s_free[t], ((gp / NS) + 1) & 1, lim, W_KW_S_FREE))) break;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
            umma_ss(tmem + t * 128, sdesc_sw128(kb0 + u * C::TILE + o, 16, 1024),
                    sdesc_sw128(qb0 + s * C::TILE + o, 16, 1024), IDESC, kk > 0);
          }
          umma_commit(&s_full[t]);
          umma_commit(&q_empty[s]);
        }
        if (!ok) break;
        umma_commit(&k_free[u]);
        ++it;
      }
      umma_commit(mma_done);                       // nothing in flight on the tensor pipe at the end
      mbar_wait(mma_done, 0, lim, W_KW_DONE);
    }
  } else if (warp >= 18) {
    // ------------------------------------------------------------ LSE rows --
    KwItem I;
    int rd = -1, n = 0, gp = -1;                   // item, pair within it, pair of the CTA
    I.n1 = 0;
    auto next = [&] {                              // the following pair; false past the last
      ++gp;
      ++n;
      while (n >= I.n1) {
        if (++rd * static_cast<int>(gridDim.x) >= p.num_items) return false;
        I = kw_item(p, rd);
        n = I.n0;
      }
      return true;
    };
    auto mine = [&] {                              // this warp's next pair
      bool more = next();
      while (more && (gp & 1) != warp - 18) more = next();
      return more;
    };
    auto load = [&](float (&v)[4]) {
      int h;
      const int i = p.by_group.divmod(n, h);
      const float* src = p.lse + (static_cast<size_t>(I.b) * p.Hq + I.hkv * G + h) * p.Lq;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = (I.i0 + i) * 128 + u * 32 + lane;
        v[u] = row < p.Lq ? src[row] : -INFINITY;
      }
    };
    float v[4], ahead[4] = {0.f, 0.f, 0.f, 0.f};
    bool more = mine();
    if (more) load(v);
    while (more) {
      const int g = gp, s = g % NR;
      more = mine();
      if (more) load(ahead);
      if (g >= NR && !mbar_wait_warp(&r_empty[s], ((g / NR) + 1) & 1, lim, W_KW_ROW_EMPTY)) break;
      float* dst = reinterpret_cast<float*>(smem + C::ROW_OFF) + s * 128;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        dst[u * 32 + lane] = v[u] == -INFINITY ? -INFINITY : -v[u] * LOG2E;    // rows without a key: their p is 0
        v[u] = ahead[u];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&r_full[s]);
    }
  } else if (warp < 16) {
    // ---------------------------------------------- one thread per key --
    const int wg = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_bits = static_cast<uint32_t>((warp & 3) * 32) << 16;
    float* sums = reinterpret_cast<float*>(smem + C::SUM_OFF);
    int gp = 0, done = 0;                          // pairs of the items before; items whose sums were joined
    bool ok = true;
    // constant pairs (the polynomial's coefficients carry the cap)
    constexpr bool CAP = (MOD & MOD_CAP) != 0, BIAS = (MOD & MOD_BIAS) != 0;
    constexpr int CW = CAP ? 16 : 32;              // queries per step
    [[maybe_unused]] f2 cscale = 0, cstep = 0, cy = 0, ck0 = 0, ck1 = 0, ck2 = 0, ck3 = 0, ck4 = 0, ck5 = 0;
    if constexpr (!CAP) cscale = f2_dup(p.scale_log2);
    if constexpr (BIAS) cstep = f2_dup(-2.f);
    if constexpr (CAP) {
      const float cap2 = p.sc.cap_log2;
      cy = f2_dup(p.sc.y_scale);
      ck0 = f2_dup(FA_TANH_C0 * cap2);
      ck1 = f2_dup(FA_TANH_C1 * cap2);
      ck2 = f2_dup(FA_TANH_C2 * cap2);
      ck3 = f2_dup(FA_TANH_C3 * cap2);
      ck4 = f2_dup(FA_TANH_C4 * cap2);
      ck5 = f2_dup(FA_TANH_C5 * cap2);
    }
    for (int rd = 0; ok && rd * static_cast<int>(gridDim.x) < p.num_items; ++rd) {
      const KwItem I = kw_item(p, rd);
      if (I.j < 0) continue;
      const int key = I.j * 128 + r;
      int kid = -1;
      if (p.sc.k_docs != nullptr && key < p.Lk) kid = p.sc.k_docs[static_cast<size_t>(I.b) * p.Lk + key];
      float a0 = 0.f, a1 = 0.f;
      for (int n = I.n0 + ((wg - gp) & 3); n < I.n1; n += 4) {
        const int g = gp + n - I.n0;
        int h;
        const int i = I.i0 + p.by_group.divmod(n, h), t = g % NS, s = g % NR, q0 = i * 128;
        // which queries see the key: causal, prefix, ragged end, documents
        uint32_t m[4];
        bool part;
        {
          int quni = -1;
          if (p.sc.q_docs != nullptr) quni = p.sc.q_meta[static_cast<size_t>(I.b) * ((p.Lq + 127) >> 7) + i].x;
          const bool docs_part = p.sc.q_docs != nullptr && (quni < 0 || quni != I.kuni);
          part = docs_part || (p.sc.causal && I.j * 128 + 127 > q0 + off && I.j * 128 + 128 > I.pre);
          const int cmin = p.sc.causal && key >= I.pre ? key - off - q0 : 0;
#pragma unroll
          for (int w4 = 0; w4 < 4; ++w4) m[w4] = ~bits_below(cmin, w4);
          if (docs_part) {
            int qid[4];
#pragma unroll
            for (int w4 = 0; w4 < 4; ++w4) {
              const int qr = q0 + w4 * 32 + lane;
              qid[w4] = qr < p.Lq ? p.sc.q_docs[static_cast<size_t>(I.b) * p.Lq + qr] : -1;
            }
            doc_bits(kid, qid, m);
          }
        }
        [[maybe_unused]] f2 cslope = 0;
        if constexpr (BIAS) cslope = f2_dup(p.sc.slopes[I.hkv * G + h] * LOG2E);
        const bool cross = (!p.sc.causal || I.pre > 0) && I.j * 128 + 127 > q0 + off;
        if (!(ok = mbar_wait_warp(&r_full[s], (g / NR) & 1, lim, W_KW_ROW) &&
                   mbar_wait_warp(&s_full[t], (g / NS) & 1, lim, W_KW_S)))
          break;
        tc_fence_after();
        const float4* row = reinterpret_cast<const float4*>(smem + C::ROW_OFF + s * 512);
        const int chunks = (min(128, p.Lq - q0) + CW - 1) / CW;
        float d0 = static_cast<float>(key - off - q0);             // distance key - query of the chunk's column 0
        f2 sum = f2_pack(a0, a1);
#pragma unroll 1
        for (int c4 = 0; c4 < chunks; ++c4) {
          uint32_t sv[CW];
          if constexpr (CAP) tmem_ld_32x32b_x16(tmem + lane_bits + t * 128 + c4 * CW, sv);
          else tmem_ld_32x32b_x32(tmem + lane_bits + t * 128 + c4 * CW, sv);
          if (c4 + 1 == chunks) { tc_fence_before(); mbar_arrive(&s_free[t]); }
          float (&x)[CW] = *reinterpret_cast<float(*)[CW]>(sv);
          const int w4 = c4 * CW >> 5;
          const uint32_t bits = (w4 == 0 ? m[0] : w4 == 1 ? m[1] : w4 == 2 ? m[2] : m[3]) >> (c4 * CW & 31);
          // x (with a cap: the tanh's arguments) to probabilities, added up.
          // GEN: with the mask and the bias' absolute value; EXACT: arguments past
          // FA_TANH_LIMIT too.
          auto add = [&](auto gen_c, auto exact_c) {
            constexpr bool GEN = decltype(gen_c)::value, EXACT = decltype(exact_c)::value;
            f2 dist = f2_pack(d0, d0 - 1.f);
#pragma unroll
            for (int c = 0; c < CW; c += 4) {
              const float4 l4 = row[c4 * CW / 4 + c / 4];               // -LSE in log2 units
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int e = c + 2 * h;
                const f2 v = f2_pack(x[e], x[e + 1]);
                f2 z, b = f2_pack(h ? l4.z : l4.x, h ? l4.w : l4.y);
                if constexpr (BIAS) {
                  f2 d = dist;
                  if constexpr (GEN) {
                    float t0, t1;
                    f2_get(d, t0, t1);
                    d = f2_pack(-fabsf(t0), -fabsf(t1));
                  }
                  b = f2_fma(d, cslope, b);
                  dist = f2_add(dist, cstep);
                }
                if constexpr (CAP) {
                  const f2 u = f2_mul(v, v);
                  f2 q = f2_fma(u, ck5, ck4);
                  q = f2_fma(q, u, ck3);
                  q = f2_fma(q, u, ck2);
                  q = f2_fma(q, u, ck1);
                  q = f2_fma(q, u, ck0);
                  z = f2_fma(v, q, b);
                  if constexpr (EXACT) {                                // each argument by itself: fa_score.cuh
                    float u0, u1, z0, z1, e0, e1;
                    f2_get(u, u0, u1);
                    f2_get(z, z0, z1);
                    f2_get(f2_fma(f2_pack(tanh_mufu(x[e]), tanh_mufu(x[e + 1])), f2_pack(p.sc.cap_log2, p.sc.cap_log2), b),
                           e0, e1);
                    constexpr float L2 = FA_TANH_LIMIT * FA_TANH_LIMIT;
                    z = f2_pack(u0 <= L2 ? z0 : e0, u1 <= L2 ? z1 : e1);
                  }
                } else {
                  z = f2_fma(v, cscale, b);
                }
                float p0, p1;
                f2_get(z, p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                if constexpr (GEN) {
                  p0 = (bits >> e) & 1u ? p0 : 0.f;
                  p1 = (bits >> (e + 1)) & 1u ? p1 : 0.f;
                }
                sum = f2_add(sum, f2_pack(p0, p1));
              }
            }
          };
          bool exact = false;
          if constexpr (CAP) {
            float umax = 0.f;
#pragma unroll
            for (int c = 0; c < CW; c += 2) {
              const f2 y = f2_mul(f2_pack(x[c], x[c + 1]), cy), u = f2_mul(y, y);
              float u0, u1;
              f2_get(y, x[c], x[c + 1]);
              f2_get(u, u0, u1);
              umax = fmax3(umax, u0, u1);
            }
            exact = __any_sync(0xffffffffu, !(umax <= FA_TANH_LIMIT * FA_TANH_LIMIT));
          }
          if (CAP && exact) add(std::true_type{}, std::true_type{});
          else if (part || (BIAS && cross)) add(std::true_type{}, std::false_type{});
          else add(std::false_type{}, std::false_type{});
          d0 -= static_cast<float>(CW);
        }
        f2_get(sum, a0, a1);
        mbar_arrive(&r_empty[s]);
      }
      if (!ok) break;
      gp += I.n1 - I.n0;
      // the warpgroups' sums of the item, joined in a fixed order
      const float mine = a0 + a1;
      if (wg > 0) {
        if (done >= 1 && !(ok = mbar_wait_warp(sum_free, (done + 1) & 1, lim, W_KW_SUM_FREE))) break;
        sums[(wg - 1) * 128 + r] = mine;
        mbar_arrive(sum_full);
      } else {
        if (!(ok = mbar_wait_warp(sum_full, done & 1, lim, W_KW_SUM))) break;
        const float total = (mine + sums[r]) + (sums[128 + r] + sums[256 + r]);
        mbar_arrive(sum_free);
        if (p.parts > 1) {
          const int nk = (p.Lk + 127) >> 7;
          const size_t at = ((static_cast<size_t>(I.part) * p.B + I.b) * p.Hkv + I.hkv) * nk * 128 + key;
          if (index_ok(at, 1, static_cast<size_t>(p.parts) * p.B * p.Hkv * nk * 128, W_IDX_KW_OUT)) p.out[at] = total;
        } else if (key < p.Lk) {
          const size_t at = (static_cast<size_t>(I.b) * p.Hkv + I.hkv) * p.ld + key;
          if (index_ok(at, 1, static_cast<size_t>(p.B) * p.Hkv * p.ld, W_IDX_KW_OUT))
            p.out[at] = p.accumulate ? p.out[at] + total : total;
        }
      }
      ++done;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The parts of each key's weight, added first to last.
__global__ void __launch_bounds__(256) kw_reduce_kernel(const float* part, float* out, int parts, int BH, int Lk, int ld,
                                                        int accumulate) {
  pdl_wait();
  const int Lp = (Lk + 127) / 128 * 128;
  const size_t n = static_cast<size_t>(BH) * Lk;
  for (size_t i = blockIdx.x * size_t(blockDim.x) + threadIdx.x; i < n; i += size_t(gridDim.x) * blockDim.x) {
    const size_t bh = i / Lk, key = i % Lk;
    float a = 0.f;
    for (int q = 0; q < parts; ++q) a += part[(size_t(q) * BH + bh) * Lp + key];
    const size_t at = bh * ld + key;
    if (!index_ok(at, 1, static_cast<size_t>(BH) * ld, W_IDX_KW_OUT)) continue;
    out[at] = accumulate ? out[at] + a : a;
  }
}

}  // namespace fa
