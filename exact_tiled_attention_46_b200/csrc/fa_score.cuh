// Score modifiers and masks shared by the scored kernels (forward, backward,
// key weights, decode).  With z = scale * q.k the score of query i and key j is
//     s = cap * tanh(z / cap)                       (when a cap is given)
//     s = s - slope_h * |i + Lk - Lq - j|           (when slopes are given)
// over the allowed pairs: j <= i + Lk - Lq or j < prefix_b (causal), and
// doc(i) = doc(j) >= 0 (documents).  The kernels work in log2 units.
#pragma once
#include <climits>
#include "sm100.cuh"
#include "tanh_poly.cuh"

namespace fa {

struct ScoreParams {
  float y_scale;           // scale / cap: raw product -> argument of the tanh
  float cap_log2;          // cap * log2(e)
  const float* slopes;     // [Hq] or nullptr
  const int* q_docs;       // [B, Lq] or nullptr
  const int* k_docs;       // [B, Lk] or nullptr
  const int* prefix;       // [B] or nullptr
  // per 128-row tile {the one document of all its rows or -1, first tile of the
  // other side that shares a document with it, one past the last, some key is
  // seen by no query (where that was asked for)}; only with documents
  const int4* q_meta;      // [B, ceil(Lq / 128)]
  const int4* k_meta;      // [B, ceil(Lk / 128)]
  int causal;
  int* counter;            // work counter of the dynamic schedule, or nullptr; zeroed beside the tile facts
};
// Kernel variants: 0 the plain kernels, else SCORED plus what the scores need.
// MOD_FINE (forward): P in two bf16 parts, and O's rounding handed out when asked for.
enum : int { MOD_NONE = 0, MOD_SCORED = 1, MOD_CAP = 2, MOD_BIAS = 4, MOD_FINE = 8 };
constexpr float LOG2E = 1.4426950408889634f;

// Prefix length of batch row b, within [0, Lk].
__device__ __forceinline__ int score_prefix(const ScoreParams& s, int b, int Lk) {
  return s.prefix != nullptr ? max(0, min(s.prefix[b], Lk)) : 0;
}

// ------------------------------------------------------------- tile facts --
// One block per (tile, batch row), query tiles first: the tile's smallest and
// largest document, then the range of the other side's tiles whose documents
// overlap that interval (exact for packed documents, which only grow along the
// row; for ids in any order the range may hold tiles without a common document,
// and the element masks decide).  Reads 4 (Lq + Lk) bytes per block out of L2:
// 3 us at L = 1000, 9 at B8 L4096 (of a forward of 500), hidden in part by the
// next kernel's start.  `unseen` (or nullptr) receives 128 bits per key tile: the
// keys that no query may see.  A warp looks its 32 keys up among the range's
// queries, 32 at a time from the first that position allows, until all are found
// (packed documents: within the first steps).
__global__ void __launch_bounds__(256) score_meta_kernel(const int* q_docs, const int* k_docs, int Lq, int Lk,
                                                         int4* q_meta, int4* k_meta, int* counter, uint32_t* zero8,
                                                         uint32_t* unseen, int causal, const int* prefix) {
  pdl_next();
  const int nq = (Lq + 127) >> 7, nk = (Lk + 127) >> 7;
  const int b = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const bool q_side = static_cast<int>(blockIdx.x) < nq;
  const int tile = q_side ? blockIdx.x : blockIdx.x - nq;
  const int* mine = q_side ? q_docs + static_cast<size_t>(b) * Lq : k_docs + static_cast<size_t>(b) * Lk;
  const int* other = q_side ? k_docs + static_cast<size_t>(b) * Lk : q_docs + static_cast<size_t>(b) * Lq;
  const int Lm = q_side ? Lq : Lk, Lo = q_side ? Lk : Lq, no = q_side ? nk : nq;
  __shared__ int s_lo[8], s_hi[8];
  // smallest and largest document of 128 rows (every lane of the warp gets them)
  auto range = [&](const int* ids, int L, int t, int& mn, int& mx, bool& neg) {
    mn = INT_MAX; mx = -1; neg = false;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int r = t * 128 + u * 32 + lane;
      if (r >= L) continue;
      const int d = ids[r];
      if (d < 0) neg = true;
      else { mn = min(mn, d); mx = max(mx, d); }
    }
    mn = __reduce_min_sync(0xffffffffu, mn);
    mx = __reduce_max_sync(0xffffffffu, mx);
    neg = __any_sync(0xffffffffu, neg);
  };
  int mn, mx;
  bool neg;
  range(mine, Lm, tile, mn, mx, neg);
  int lo = INT_MAX, hi = 0;
  if (mx >= 0)
#pragma unroll 4
    for (int t = warp; t < no; t += 8) {
      int on, ox;
      bool og;
      range(other, Lo, t, on, ox, og);
      if (on <= mx && mn <= ox) { lo = min(lo, t); hi = t + 1; }
    }
  if (lane == 0) { s_lo[warp] = lo; s_hi[warp] = hi; }
  __syncthreads();
  for (int w = 0; w < 8; ++w) { lo = min(lo, s_lo[w]); hi = max(hi, s_hi[w]); }
  if (lo > hi) lo = hi = 0;
  bool miss = false;                             // this thread's key is seen by no query
  if (unseen != nullptr && !q_side) {
    if (warp < 4) {
      const int key = tile * 128 + warp * 32 + lane, kid = key < Lk ? mine[key] : -1;
      const int pre = prefix != nullptr ? prefix[b] : 0;
      const int from = causal && key >= pre ? max(0, key - (Lk - Lq)) : 0;   // first query that position allows
      const bool live = kid >= 0;
      bool seen = key >= Lk;
      const int q1 = min(hi * 128, Lq);
      for (int q0 = max(lo * 128, __reduce_min_sync(0xffffffffu, live ? from : INT_MAX) & ~31); q0 < q1; q0 += 32) {
        if (__all_sync(0xffffffffu, seen || !live)) break;
        const int qd = q0 + lane < q1 ? other[q0 + lane] : -1;
#pragma unroll
        for (int u = 0; u < 32; ++u) {
          const int d = __shfl_sync(0xffffffffu, qd, u);
          seen |= live && d == kid && q0 + u >= from;
        }
      }
      miss = !seen;
      const uint32_t bits = __ballot_sync(0xffffffffu, miss);
      if (lane == 0) unseen[(static_cast<size_t>(b) * nk + tile) * 4 + warp] = bits;
    }
    miss = __syncthreads_or(miss);
  }
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0 && b == 0) {
      *counter = 0;
      if (zero8 != nullptr)                      // eight words that the caller's next kernel adds to
        for (int i = 0; i < 8; ++i) zero8[i] = 0;
    }
    (q_side ? q_meta + static_cast<size_t>(b) * nq : k_meta + static_cast<size_t>(b) * nk)[tile] =
        make_int4(mn == mx && !neg ? mn : -1, lo, hi, miss ? 1 : 0);
  }
}

// ------------------------------------------------------------------ masks --
// Bits c of word w (columns 32 w + c) with 32 w + c < lim.
__device__ __forceinline__ uint32_t bits_below(int lim, int w) {
  const int n = lim - 32 * w;
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}
// Document masks of a tile: lane L's row holds document `id`, and other[w] is
// the document of column 32 w + L.  Every distinct document of the warp's rows
// is matched against all columns by one ballot per word.
template <int W>
__device__ __forceinline__ void doc_bits(int id, const int (&other)[W], uint32_t (&m)[W]) {
  uint32_t d[W];
#pragma unroll
  for (int w = 0; w < W; ++w) d[w] = 0u;
  uint32_t todo = __ballot_sync(0xffffffffu, id >= 0);
  while (todo) {
    const int cur = __shfl_sync(0xffffffffu, id, __ffs(todo) - 1);
    const bool mine = id == cur;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const uint32_t hit = __ballot_sync(0xffffffffu, other[w] == cur);
      if (mine) d[w] = hit;
    }
    todo &= ~__ballot_sync(0xffffffffu, mine);
  }
#pragma unroll
  for (int w = 0; w < W; ++w) m[w] &= d[w];
}

// Is there an inf or NaN among bf16 values?  x * 0 + a keeps a NaN once any x is
// not finite.
__device__ __forceinline__ __nv_bfloat162 poison8(const uint4& w, __nv_bfloat162 a) {
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.x), zero, a);
  a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.y), zero, a);
  a = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.z), zero, a);
  return __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&w.w), zero, a);
}
__device__ __forceinline__ bool is_nan2(__nv_bfloat162 a) { return __hisnan(a.x) || __hisnan(a.y); }

// -------------------------------------------------------------------- cap --
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh for any argument on the MUFU unit: 1 - 2 / (1 + e^(2y)), absolute error
// about 2^-22 (two MUFU operations).  The kernels take it for arguments beyond
// FA_TANH_LIMIT, where that is half a step of fp32 relative to the value, and the
// polynomial below within.  Each argument decides for itself: what else stands in
// the tile, masked or of another row, changes no bit of a score.  (A warp without
// any argument beyond the limit skips the MUFU form.)
__device__ __forceinline__ float tanh_mufu(float y) {
  return fmaf(-2.f, rcp_approx(1.f + ex2_approx(2.f * LOG2E * y)), 1.f);
}
// tanh of two arguments within FA_TANH_LIMIT on the FMA pipe: y p(y^2), packed fp32.
__device__ __forceinline__ void tanh_poly2(float y0, float y1, float& t0, float& t1) {
  float u0, u1, p0, p1;
  ffma2(u0, u1, y0, y1, y0, y1, 0.f, 0.f);
  ffma2(p0, p1, u0, u1, FA_TANH_C5, FA_TANH_C5, FA_TANH_C4, FA_TANH_C4);
  ffma2(p0, p1, p0, p1, u0, u1, FA_TANH_C3, FA_TANH_C3);
  ffma2(p0, p1, p0, p1, u0, u1, FA_TANH_C2, FA_TANH_C2);
  ffma2(p0, p1, p0, p1, u0, u1, FA_TANH_C1, FA_TANH_C1);
  ffma2(p0, p1, p0, p1, u0, u1, FA_TANH_C0, FA_TANH_C0);
  ffma2(t0, t1, y0, y1, p0, p1, 0.f, 0.f);
}
// tanh of any two arguments (a NaN gives a NaN).
__device__ __forceinline__ void tanh_any2(float y0, float y1, float& t0, float& t1) {
  tanh_poly2(y0, y1, t0, t1);
  t0 = fabsf(y0) <= FA_TANH_LIMIT ? t0 : tanh_mufu(y0);
  t1 = fabsf(y1) <= FA_TANH_LIMIT ? t1 : tanh_mufu(y1);
}

// Raw products x[0..16) to t = tanh(x * y_scale), in place.  The polynomial costs
// 8 packed FMAs per pair, the other form 4 MUFU operations besides.
__device__ __forceinline__ void cap_tile(float (&x)[16], float ysc) {
  float a0 = 0.f, a1 = 0.f;
#pragma unroll
  for (int c = 0; c < 16; c += 4) {
    a0 = fmaxf(a0, fmaxf(fabsf(x[c]), fabsf(x[c + 1])));
    a1 = fmaxf(a1, fmaxf(fabsf(x[c + 2]), fabsf(x[c + 3])));
  }
  if (!__any_sync(0xffffffffu, !(fmaxf(a0, a1) * ysc <= FA_TANH_LIMIT))) {
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      float y0, y1;
      ffma2(y0, y1, x[c], x[c + 1], ysc, ysc, 0.f, 0.f);
      tanh_poly2(y0, y1, x[c], x[c + 1]);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 16; c += 2) {
      float y0, y1;
      ffma2(y0, y1, x[c], x[c + 1], ysc, ysc, 0.f, 0.f);
      tanh_any2(y0, y1, x[c], x[c + 1]);
    }
  }
}

}  // namespace fa
