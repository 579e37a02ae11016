// Prefill forward: exact softmax(Q K^T * scale) V, tile by tile with an online
// softmax ("FlashAttention Explained: How AI Models Process Attention Faster
// and Use Less Memory", sections "1. Tiling", "3. Online Softmax" and "Fused
// Computation"; "Flash Attention Explained: Same Maths, Far Less Memory",
// section "The idea: never materialise the matrix").  The score matrix lives
// only in tensor memory; Q is read and O/LSE written once, K and V once per
// work item (the re-reads of a head's K and V by its other items hit L2).
//
// The grid is persistent (at most one CTA per SM).  A work item is a pair of
// 128-row query tiles of one (batch, head); a CTA takes its items one after the
// other and, for each, walks the key tiles of the kv head:
//   warp 8      TMA producer: the item's Q tiles (each slot refilled once the
//               previous item's last S on it is done), then K_j, V_j into a
//               slot ring that runs on from item to item
//   warp 9      MMA issuer:   S_t = Q_t K_j^T into TMEM, O_t += P_t V_j
//   warps 0-3   softmax for query tile 0, warps 4-7 for query tile 1: one
//               thread per query row; causal / ragged mask; running max m and
//               running sum l in log2 units; P (bf16) written over S in TMEM;
//               O rescaled in TMEM only when the max grows by more than TAU;
//               epilogue O / l and LSE.
//   warp 10     allocates / frees the 512 TMEM columns; warp 11 idles (scored
//               variants: it looks V tiles over, below).
// Registers: the block is launched with FWD_LAUNCH_REGS per thread (3 warps per
// SM sub-partition); the control warpgroup (warps 8-11) gives registers back
// (setmaxnreg.dec to FwdRegs::CTRL) and the two softmax warpgroups take them
// (setmaxnreg.inc to FwdRegs::SOFTMAX).  The split sums to exactly the launch
// allocation: 2 * 224 + 56 = 3 * 168 registers per lane slot.
// TMEM columns: S_0 [0,128), S_1 [128,256), O_0 [256,256+D), O_1 after it.
//
// The scored variants (MOD != 0) add a tanh cap, a distance bias, documents and
// a prefix to the scores (fa_score.cuh).  Their key tiles run from the first to
// the last one that shares a document with the item's queries.  A tile's mask is
// one 128-bit word per query row, put together while the warp waits for S.
// Masked probabilities are 0, but 0 * NaN is not: in a tile that any of the
// item's rows sees in part, warp 11 looks for V rows that hold an inf or NaN
// before the product reads them, clears them, and names them to the softmax
// warps; a row that may see one of them ends as NaN, the others are untouched.
// With nothing changed the scored kernel takes 104 us where the plain one takes
// 86 (causal B4 H16 L2048 D128); without warp 11's code it takes 10 less, its
// waits and looks alone cost nothing.  P in two parts adds 28 us (the second set
// of products and stores), a cap 16 to that (its polynomial), a bias 7, o_lo 7
// (2 with a cap).  Floors there: 41 us of products (62 in two parts), 29 of
// exponentials; what bounds all of them is the chain from one S through P to the
// next on two warps per sub-partition.
// MOD_FINE keeps P in two bf16 parts (the second takes the other half of S's
// columns and a second set of P.V products), so that O is off by its own rounding
// alone: relative error 1.66e-3 in bf16 where one part gives 1.9e-3, for 157 us
// instead of 128 (cap, B4 H16 L2048 D128) and 900 instead of 661 (bias and prefix,
// Hq32 Hkv8 L8191 D128).  Every scored call takes it but the one that changes
// nothing, which is fa_fwd_ex bit for bit.  With o_lo it writes, beside the bf16 O,
// what that rounding took off: the gradient's Delta = dO.O subtracts from dP
// values close to it, and an O rounded to bf16 costs dq and dk half again of what
// their own rounding does (train step B2 Hq16 Hkv4 L2048 D128, scores peaked:
// relative error 2.8e-3 where the outputs' rounding alone gives 1.7e-3).
#pragma once
#include "sm100.cuh"
#include "exp2_poly.cuh"
#include "fa_score.cuh"

namespace fa {

struct FwdParams {
  void* o;                 // [B, Lq, Hq, D] bf16 or fp32
  float* lse;              // [B, Hq, Lq] or nullptr
  int B, Hq, Hkv, Lq, Lk;
  int num_pairs;           // items per (batch, head): ceil(Lq / 256), scored ceil(Lq / item_rows)
  float scale_log2;        // scale * log2(e) (e4m3 inputs: times the Q and K scales)
  float o_scale;           // multiplies O (e4m3 inputs: the V scale; else 1)
  int o_fp32;
  uint64_t wait_limit_ns;
  ScoreParams sc;          // scored variants only
  int item_rows;           // scored: query rows per item, 256 or 128 (no second query tile)
  uint16_t* o_lo;          // MOD_FINE: [B, Lq, Hq, D] bf16, O minus its rounding, or nullptr
};

// FP8: Q, K, V are e4m3 (one byte per element) and both products run as
// kind::f8f6f4 (D = 128 only: one 128-byte swizzle column per row).
template <int D, bool FP8 = false, int MOD = MOD_NONE>
struct FwdCfg {  // scored variants: a two-entry item queue and the V tiles' state besides
  static constexpr int ES = FP8 ? 1 : 2;               // bytes per input element
  static constexpr int TILE_BYTES = 128 * D * ES;      // one 128-row tile
  static constexpr int KB = D * ES / 128;              // 128-byte column blocks per row (one TMA box each)
  static constexpr int NS = (TILE_BYTES == 32768) ? 4 : 8;   // K/V slots
  static constexpr int Q_OFF = 0;
  static constexpr int KV_OFF = 2 * TILE_BYTES;
  static constexpr int BAR_OFF = KV_OFF + NS * TILE_BYTES;
  static constexpr int NBARS = 2 + 2 + 2 * NS + 2 + 2 + 2 + 1 + (MOD ? NS + 4 : 0);
  static constexpr int BAD_OFF = BAR_OFF + (NBARS * 8 + 31) / 16 * 16;   // scored: per slot, 128 bits of unusable V rows
  static constexpr int ITEM_OFF = BAD_OFF + NS * 16;   // scored: item queue
  static constexpr int SMEM_BYTES = MOD ? ITEM_OFF + 16 + 1024 : BAR_OFF + NBARS * 8 + 16 + 1024;
  static constexpr int THREADS = 384;
};

// The running max m is a reference only: any m gives the same exact result.
// A tile is first exponentiated against the current m; if no lane's tile sum
// exceeds 2^FWD_FAST_LOG2 (so every p <= 2^16, a range bf16 and the fp32
// accumulators hold with unchanged relative precision), that is the tile's P.
// Otherwise (and on a row's first tile) the tile max is taken, m moves to it
// when it grows by more than FWD_TAU, O and the sums are rescaled in place, and
// P is recomputed.
constexpr float FWD_TAU = 8.0f;
// Caps (log2 units; 50.6 in score units) up to which no largest score is looked for.
constexpr float FWD_CAP_FREE = 73.0f, FWD_CAP_ROOM = 24.0f;
constexpr int FWD_LAUNCH_REGS = 168;
// With a cap the scores come 32 columns at a time and the softmax warps need
// fewer registers, while the thread that issues the products gains from more
// (capped prefill B4 H16 L2048 D128: 149 us with 208 and 88, 152 with 224 and
// 56, 154 with 192 and 120; Hq32 Hkv8 L8192: 940, 940, 963); the other variants
// hold a whole row of S and spill below 224 (a bias: 140 us, 142 with 208).
template <int MOD>
struct FwdRegs {
  static constexpr int SOFTMAX = (MOD & MOD_CAP) ? 208 : 224, CTRL = (MOD & MOD_CAP) ? 88 : 56;
  static_assert(2 * SOFTMAX + CTRL == 3 * FWD_LAUNCH_REGS, "register split must match the launch");
};
constexpr float FWD_FAST_LIMIT = 65536.0f;
// Every FWD_POLY_PERIOD-th pair of an unmasked tile can be exponentiated on the
// FMA pipe (exp2_poly2) instead of the MUFU unit; 0 turns this off.  Measured
// against a share of 1/3 on the causal prefill (B4 H16 L2048 D128) and long GQA
// (B1 Hq32 Hkv8 L16384 D128) workloads: 1/2 gave -4% / -1%, 1/4 +2% / +3.5%,
// 1/8 +3% / +5%, none +3% / +7%.  The softmax warps here are bound by their
// issue slots rather than by the MUFU rate, so the longer polynomial sequence
// does not pay.
constexpr int FWD_POLY_PERIOD = 0;
__host__ __device__ constexpr bool fwd_poly_pair(int i) {
  return FWD_POLY_PERIOD > 0 && (i % (FWD_POLY_PERIOD > 0 ? FWD_POLY_PERIOD : 1)) == FWD_POLY_PERIOD - 1;
}

// 2^x for two lanes on the FMA pipe: x = j + f with j = round(x), f in
// [-1/2, 1/2]; 2^f by the fitted polynomial (exp2_poly.cuh, Horner on packed
// fp32); 2^j added into the exponent field.  x is clamped to [-126, 127]:
// below, the result is a tiny positive number (not 0) far below 2^-126, so
// callers use it only where no entry is masked; above, it stays the finite
// 2^127 (never a wrapped exponent), which still trips the fast path's sum
// limit.  Relative error <= FA_EXP2_MAX_REL_ERR + fp32 rounding in the range.
__device__ __forceinline__ void exp2_poly2(float x0, float x1, float& p0, float& p1) {
  x0 = fminf(fmaxf(x0, -126.f), 127.f);
  x1 = fminf(fmaxf(x1, -126.f), 127.f);
  constexpr float RND = 12582912.f;                  // 1.5 * 2^23: x + RND rounds x to an integer
  float t0, t1, r0, r1, f0, f1, q0, q1;
  fadd2(t0, t1, x0, x1, RND, RND);
  fadd2(r0, r1, t0, t1, -RND, -RND);                 // round(x) as a float
  ffma2(f0, f1, r0, r1, -1.f, -1.f, x0, x1);         // f = x - round(x)
  ffma2(q0, q1, f0, f1, FA_EXP2_C3, FA_EXP2_C3, FA_EXP2_C2, FA_EXP2_C2);
  ffma2(q0, q1, q0, q1, f0, f1, FA_EXP2_C1, FA_EXP2_C1);
  ffma2(q0, q1, q0, q1, f0, f1, FA_EXP2_C0, FA_EXP2_C0);
  // the low mantissa bits of t hold round(x) (two's complement); << 23 moves it to the exponent
  p0 = __uint_as_float(__float_as_uint(q0) + (__float_as_uint(t0) << 23));
  p1 = __uint_as_float(__float_as_uint(q1) + (__float_as_uint(t1) << 23));
}

// The e4m3 path stores P scaled by 2^FWD_F8_P_LOG2 against the reference max
// and moves the reference whenever a tile max exceeds it by more than
// FWD_F8_TAU, so every stored value is at most 2^(8 + 0.75) = 431 (e4m3's
// largest finite value is 448) and values down to 2^-17 of the row's largest
// stay representable.
constexpr float FWD_F8_P_LOG2 = 8.0f, FWD_F8_TAU = 0.75f;

enum : uint32_t {
  W_FWD_Q = 0x101, W_FWD_KV_EMPTY = 0x102, W_FWD_KV_FULL = 0x103, W_FWD_P = 0x104,
  W_FWD_S = 0x105, W_FWD_O = 0x106, W_FWD_DONE = 0x107, W_FWD_DRAIN = 0x108, W_FWD_Q_EMPTY = 0x109,
  W_FWD_V_OK = 0x10a, W_FWD_ITEM = 0x10b, W_FWD_ITEM_EMPTY = 0x10c
};

// One work item is a pair of 128-row query tiles of one (batch, head).  Items
// are numbered heaviest first (causal work grows with the pair index); the grid
// is persistent (at most one CTA per SM) and CTA c takes, in round r, item
// r * G + c (r even) or r * G + G - 1 - c (r odd), a boustrophedon order that
// evens out the causal work across CTAs.
struct FwdItem {
  int b, h, hkv, q0, n_t0, n_t1, n;
  // scored: query tile t takes part in steps [s_t, n_t) of the item's n (the
  // plain kernels: [0, n_t)); step i is key tile fwd_tile<MOD>(I, i)
  int s_t0, s_t1, j0;
  int pre;                 // scored: prefix length
  int part0, part1;        // scored: first key tile that query tile 0 / 1 sees in part by position alone
  int uni0, uni1;          // scored: the one document of all rows of query tile 0 / 1, or -1
};
// With a distance bias the key tiles are walked from the last to the first: a
// row's nearest keys then set its reference max, and the tiles after them stay
// below it (first to last, a steep slope raises the max in every tile, and each
// raise costs a second exponential pass and a rescale of O).
template <int MOD>
__device__ __forceinline__ int fwd_tile(const FwdItem& I, int step) {
  return (MOD & MOD_BIAS) ? I.j0 - step : MOD != MOD_NONE ? I.j0 + step : step;
}
template <bool CAUSAL, int MOD = MOD_NONE>
__device__ __forceinline__ FwdItem fwd_item(const FwdParams& p, int w) {
  FwdItem I;
  const int bh_count = p.B * p.Hq;
  const int pair = p.num_pairs - 1 - w / bh_count;
  const int bh = w % bh_count;
  I.b = bh / p.Hq;
  I.h = bh % p.Hq;
  I.hkv = I.h / (p.Hq / p.Hkv);
  I.q0 = pair * (MOD == MOD_NONE ? 256 : p.item_rows);
  const int off = p.Lk - p.Lq;
  const int nk_all = (p.Lk + 127) >> 7;
  I.s_t0 = I.s_t1 = I.j0 = 0;
  if constexpr (MOD != MOD_NONE) {
    // key tiles [lo, hi) of each query tile
    const ScoreParams& sc = p.sc;
    I.pre = sc.causal ? score_prefix(sc, I.b, p.Lk) : 0;
    int lo[2], hi[2], uni[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r0 = t * 128 < p.item_rows ? I.q0 + t * 128 : p.Lq;
      lo[t] = 0;
      hi[t] = r0 < p.Lq ? nk_all : 0;
      uni[t] = -1;
      if (r0 < p.Lq && sc.causal) {
        const int lim_keys = max(min(r0 + 127, p.Lq - 1) + off + 1, I.pre);
        hi[t] = lim_keys <= 0 ? 0 : min(nk_all, (lim_keys + 127) >> 7);
      }
      if (r0 < p.Lq && sc.q_docs != nullptr) {
        const int4 m = sc.q_meta[static_cast<size_t>(I.b) * ((p.Lq + 127) >> 7) + (r0 >> 7)];
        uni[t] = m.x;
        lo[t] = m.y;
        hi[t] = min(hi[t], m.z);
      }
      if (lo[t] >= hi[t]) { lo[t] = INT_MAX; hi[t] = 0; }
      // tiles before `part` hold only keys that every row of the tile sees
      const int seen = sc.causal ? min(p.Lk, max(max(r0 + off + 1, 0), I.pre)) : p.Lk;
      (t ? I.part1 : I.part0) = seen >> 7;
    }
    const int first = min(lo[0], lo[1]), last = max(hi[0], hi[1]);
    constexpr bool DOWN = (MOD & MOD_BIAS) != 0;
    I.j0 = DOWN ? last - 1 : first;
    I.s_t0 = hi[0] == 0 ? 0 : DOWN ? last - hi[0] : lo[0] - first;
    I.n_t0 = hi[0] == 0 ? 0 : DOWN ? last - lo[0] : hi[0] - first;
    I.s_t1 = hi[1] == 0 ? 0 : DOWN ? last - hi[1] : lo[1] - first;
    I.n_t1 = hi[1] == 0 ? 0 : DOWN ? last - lo[1] : hi[1] - first;
    I.n = max(I.n_t0, I.n_t1);
    I.uni0 = uni[0];
    I.uni1 = uni[1];
  } else {
    int nt[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r0 = I.q0 + t * 128;
      if (r0 >= p.Lq) {
        nt[t] = 0;
      } else if (!CAUSAL) {
        nt[t] = nk_all;
      } else {
        const int lim_keys = min(r0 + 127, p.Lq - 1) + off + 1;   // keys < lim_keys for the last row
        nt[t] = lim_keys <= 0 ? 0 : min(nk_all, (lim_keys + 127) >> 7);
      }
    }
    I.n_t0 = nt[0];
    I.n_t1 = nt[1];
    I.n = max(nt[0], nt[1]);
  }
  return I;
}
__device__ __forceinline__ int fwd_item_index(int r) {
  const int G = static_cast<int>(gridDim.x);
  return r * G + ((r & 1) ? (G - 1 - static_cast<int>(blockIdx.x)) : static_cast<int>(blockIdx.x));
}

// Scored variants: may some row of query tile t not see some key of tile j?
// kuni: the one document of all the key tile's rows, or -1.
__device__ __forceinline__ bool fwd_tile_masked(const FwdParams& p, const FwdItem& I, int t, int j, int kuni) {
  if (j >= (t ? I.part1 : I.part0)) return true;
  const int uni = t ? I.uni1 : I.uni0;
  return p.sc.q_docs != nullptr && (uni < 0 || uni != kuni);
}
__device__ __forceinline__ int fwd_key_doc(const FwdParams& p, int b, int j) {
  const int nk = (p.Lk + 127) >> 7;
  return p.sc.q_docs != nullptr && j < nk ? p.sc.k_meta[static_cast<size_t>(b) * nk + j].x : -1;
}

// Scored variants, one warp: clears the rows of a 128-row V tile (bf16, 128-byte
// column blocks of 16 KB) that hold an inf or NaN and writes their bits to
// bad[0..4).  One pass tells whether there are any; only then are the rows told
// apart.
template <int D>
__device__ __forceinline__ void fwd_clean_v(uint8_t* tile, uint32_t* bad) {
  const int lane = threadIdx.x & 31;
  const uint4* t4 = reinterpret_cast<const uint4*>(tile);
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.f);
  __nv_bfloat162 acc = zero, acc2 = zero;
#pragma unroll 4
  for (int c = lane; c < 128 * D * 2 / 16; c += 64) {
    acc = poison8(t4[c], acc);
    acc2 = poison8(t4[c + 32], acc2);
  }
  uint32_t word = 0;
  if (__any_sync(0xffffffffu, is_nan2(acc) || is_nan2(acc2))) {
    for (int w = 0; w < 4; ++w) {
      uint4* row = reinterpret_cast<uint4*>(tile + (w * 32 + lane) * 128);
      __nv_bfloat162 a = zero;
      for (int kb = 0; kb < D / 64; ++kb)
        for (int c = 0; c < 8; ++c) a = poison8(row[kb * 1024 + c], a);
      const bool b = is_nan2(a);
      if (b)
        for (int kb = 0; kb < D / 64; ++kb)
          for (int c = 0; c < 8; ++c) row[kb * 1024 + c] = make_uint4(0u, 0u, 0u, 0u);
      const uint32_t bits = __ballot_sync(0xffffffffu, b);
      if (lane == w) word = bits;
    }
    fence_proxy_async_smem();
  }
  if (lane < 4) bad[lane] = word;
}

// Distance from column `at` (any value) to the nearest set bit of m; -1 when none is set.
__device__ __forceinline__ int nearest_bit(const uint32_t (&m)[4], int at) {
  int best = 1 << 30;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int a = at - 32 * w;                     // column within this word
    if (m[w] == 0u) continue;
    if (a <= 0) {
      best = min(best, __ffs(m[w]) - 1 - a);
    } else if (a >= 31) {
      best = min(best, a - (31 - __clz(m[w])));
    } else {
      const uint32_t low = m[w] & ((2u << a) - 1u), high = m[w] >> a;
      if (low) best = min(best, a - (31 - __clz(low)));
      if (high) best = min(best, __ffs(high) - 1);
    }
  }
  return best == 1 << 30 ? -1 : best;
}

template <int D, bool CAUSAL, bool FP8 = false, int MOD = MOD_NONE>
__global__ void __launch_bounds__(384, 1)
fwd_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
           const __grid_constant__ CUtensorMap tm_v, const FwdParams p) {
  static_assert(!FP8 || D == 128, "the e4m3 path is built for D = 128");
  static_assert(MOD == MOD_NONE || (CAUSAL && !FP8), "the scored variants are bf16 and take the mask at run time");
  static_assert(!(MOD & (MOD_CAP | MOD_BIAS)) || (MOD & MOD_FINE), "changed scores keep P in two parts");
  using C = FwdCfg<D, FP8, MOD>;
  constexpr int NS = C::NS;
  constexpr int KB = C::KB;                        // 128-byte column blocks per row
  constexpr int BOX_COLS = 128 / C::ES;            // elements per 128-byte block
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);
  uint64_t* q_full = bars;                         // [2] Q tile t landed
  uint64_t* q_empty = q_full + 2;                  // [2] last S of Q tile t done
  uint64_t* kv_full = q_empty + 2;                 // [NS]
  uint64_t* kv_empty = kv_full + NS;               // [NS]
  uint64_t* s_full = kv_empty + NS;                // [2]
  uint64_t* p_full = s_full + 2;                   // [2]
  uint64_t* o_full = p_full + 2;                   // [2]
  uint64_t* mma_done = o_full + 2;
  uint64_t* v_ok = mma_done + 1;                   // [NS] scored: the V tile was looked over
  uint64_t* item_full = v_ok + NS;                 // [2] scored: an item number was posted
  uint64_t* item_empty = item_full + 2;            // [2] and every role has read it
  volatile int* item_w = reinterpret_cast<volatile int*>(smem + C::ITEM_OFF);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(bars + C::NBARS);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t lim = p.wait_limit_ns;
  const int G = static_cast<int>(gridDim.x);
  const int num_items = p.num_pairs * p.B * p.Hq;
  const int off = p.Lk - p.Lq;                     // bottom-right causal alignment

  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&q_full[t], 1); mbar_init(&q_empty[t], 1);
      mbar_init(&s_full[t], 1); mbar_init(&p_full[t], 128); mbar_init(&o_full[t], 1);
    }
    for (int i = 0; i < NS; ++i) { mbar_init(&kv_full[i], 1); mbar_init(&kv_empty[i], 1); }
    mbar_init(mma_done, 1);
    if constexpr (MOD != MOD_NONE) {
      for (int i = 0; i < NS; ++i) mbar_init(&v_ok[i], 1);
      // readers of the queue: the MMA thread, lane 0 of warp 11 and of the eight softmax warps
      for (int u = 0; u < 2; ++u) { mbar_init(&item_full[u], 1); mbar_init(&item_empty[u], 10); }
    }
    fence_mbar_init();
  }
  if (warp == 10) { tmem_alloc(tmem_holder, 512); tmem_relinquish(); }
  if (warp == 8 && lane == 0) { tma_prefetch_desc(&tm_q); tma_prefetch_desc(&tm_k); tma_prefetch_desc(&tm_v); }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_holder;
  if constexpr (MOD != MOD_NONE) pdl_wait();       // the tile facts of the documents

  // Scored: the r-th item that the producer posted; false (and `more` cleared)
  // after the last one.
  [[maybe_unused]] auto take = [&](int r, int& w, bool& ok, bool& more, bool whole_warp) {
    const int qs = r & 1;
    ok = whole_warp ? mbar_wait_warp(&item_full[qs], (r >> 1) & 1, lim, W_FWD_ITEM)
                    : mbar_wait(&item_full[qs], (r >> 1) & 1, lim, W_FWD_ITEM);
    w = ok ? item_w[qs] : -1;
    if (whole_warp) __syncwarp();
    if (ok && (!whole_warp || lane == 0)) mbar_arrive(&item_empty[qs]);
    more = w >= 0;
    return more;
  };

  if (warp >= 8) {
  setmaxnreg_dec<FwdRegs<MOD>::CTRL>();
  if (warp == 8) {
    // ------------------------------------------------------------ producer --
    if (lane == 0) {
      int it = 0;                                  // K/V ring loads issued
      uint32_t q_loaded = 0, q_par = 0;            // bit t: Q slot t loaded before / parity of its loads
      bool ok = true;
      for (int r = 0; ok; ++r) {
        int w;
        if constexpr (MOD == MOD_NONE) {
          if (r * G >= num_items) break;
          w = fwd_item_index(r);
          if (w >= num_items) continue;
        } else {
          // from the launch's counter where documents make the items' weights
          // unforeseeable, else in the fixed order (its last round may be short)
          w = p.sc.counter != nullptr ? atomicAdd(p.sc.counter, 1) : r * G < num_items ? fwd_item_index(r) : num_items;
          if (w >= num_items) w = -1;
          if (r >= 2 && !(ok = mbar_wait(&item_empty[r & 1], ((r >> 1) + 1) & 1, lim, W_FWD_ITEM_EMPTY))) break;
          item_w[r & 1] = w;
          mbar_arrive(&item_full[r & 1]);          // release: the readers' wait sees the number
          if (w < 0) break;
        }
        const FwdItem I = fwd_item<CAUSAL, MOD>(p, w);
        if (I.n == 0) continue;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          if ((t ? I.n_t1 : I.n_t0) == 0) continue;
          // wait for the previous item's last S on this slot (phase = loads so far - 1)
          if (((q_loaded >> t) & 1u) && !(ok = mbar_wait(&q_empty[t], ((q_par >> t) & 1u) ^ 1u, lim, W_FWD_Q_EMPTY))) break;
          mbar_arrive_expect_tx(&q_full[t], C::TILE_BYTES);
          for (int kb = 0; kb < KB; ++kb)
            tma_load_4d(smem + C::Q_OFF + t * C::TILE_BYTES + kb * 16384, &tm_q, &q_full[t], kb * BOX_COLS, I.h,
                        I.q0 + t * 128, I.b);
          q_loaded |= 1u << t;
          q_par ^= 1u << t;
        }
        for (int i = 0; ok && i < 2 * I.n; ++i) {
          const int slot = it % NS;
          if (it >= NS && !(ok = mbar_wait(&kv_empty[slot], ((it / NS) + 1) & 1, lim, W_FWD_KV_EMPTY))) break;
          mbar_arrive_expect_tx(&kv_full[slot], C::TILE_BYTES);
          const CUtensorMap* m = (i & 1) ? &tm_v : &tm_k;
          uint8_t* dst = smem + C::KV_OFF + slot * C::TILE_BYTES;
          for (int kb = 0; kb < KB; ++kb)
            tma_load_4d(dst + kb * 16384, m, &kv_full[slot], kb * BOX_COLS, I.hkv, fwd_tile<MOD>(I, i >> 1) * 128, I.b);
          ++it;
        }
      }
      // the CTA may not exit with copies in flight: wait for the last loads
      for (int t = 0; t < 2; ++t)
        if ((q_loaded >> t) & 1u) mbar_wait(&q_full[t], ((q_par >> t) & 1u) ^ 1u, lim, W_FWD_DRAIN);
      for (int i = max(0, it - NS); i < it; ++i) mbar_wait(&kv_full[i % NS], (i / NS) & 1, lim, W_FWD_DRAIN);
    }
  } else if (warp == 9) {
    // ----------------------------------------------------------------- MMA --
    if (lane == 0) {
      constexpr uint32_t IDESC_S = FP8 ? idesc_e4m3_f32(128, 128, false, false) : idesc_bf16_f32(128, 128, false, false);
      constexpr uint32_t IDESC_O = FP8 ? idesc_e4m3_f32(128, D, false, true) : idesc_bf16_f32(128, D, false, true);
      // every instruction consumes 32 bytes of K: 16 bf16 or 32 e4m3 elements
      constexpr int KS_S = D * C::ES / 32, KS_PV = 128 * C::ES / 32;
      const uint32_t q_base = smem_u32(smem + C::Q_OFF);
      const uint32_t kv_base = smem_u32(smem + C::KV_OFF);
      auto issue_s = [&](int t, int slot) {
        const uint32_t qa = q_base + t * C::TILE_BYTES, ka = kv_base + slot * C::TILE_BYTES;
#pragma unroll
        for (int kk = 0; kk < KS_S; ++kk) {
          const uint32_t o = (kk >> 2) * 16384 + (kk & 3) * 32;
          if constexpr (FP8)
            umma_ss_f8(tmem + t * 128, sdesc_sw128(qa + o, 16, 1024), sdesc_sw128(ka + o, 16, 1024), IDESC_S, kk > 0);
          else
            umma_ss(tmem + t * 128, sdesc_sw128(qa + o, 16, 1024), sdesc_sw128(ka + o, 16, 1024), IDESC_S, kk > 0);
        }
      };
      // P's columns of keys 16 kk .. 16 kk + 15: packed from column 0, or (capped
      // scores, formed 32 columns at a time) at the start of their own 32 columns
      auto p_col = [](int kk) { return (MOD & MOD_CAP) ? (kk >> 1) * 32 + (kk & 1) * 8 : kk * 8; };
      auto issue_pv = [&](int t, int slot, bool acc) {
        const uint32_t va = kv_base + slot * C::TILE_BYTES;
        // P (K = 128 keys) from TMEM, 8 columns per instruction; V MN-major,
        // 32 bytes of keys (16 or 32 rows of 128 bytes) per instruction
#pragma unroll
        for (int kk = 0; kk < KS_PV; ++kk) {
          if constexpr (FP8)
            umma_ts_f8(tmem + 256 + t * D, tmem + t * 128 + kk * 8, sdesc_sw128(va + kk * 4096, 16384, 1024), IDESC_O,
                       (acc || kk > 0) ? 1u : 0u);
          else
            umma_ts(tmem + 256 + t * D, tmem + t * 128 + p_col(kk), sdesc_sw128(va + kk * 2048, 16384, 1024), IDESC_O,
                    (acc || kk > 0) ? 1u : 0u);
        }
        if constexpr ((MOD & MOD_FINE) != 0) {     // the second part of P, in the other half of S's columns
#pragma unroll
          for (int kk = 0; kk < KS_PV; ++kk)
            umma_ts(tmem + 256 + t * D, tmem + t * 128 + p_col(kk) + ((MOD & MOD_CAP) ? 16 : 64),
                    sdesc_sw128(va + kk * 2048, 16384, 1024), IDESC_O, 1u);
        }
      };
      auto wait_item = [&](int i) { return mbar_wait(&kv_full[i % NS], (i / NS) & 1, lim, W_FWD_KV_FULL); };
      // V tiles (odd ring entries; the ring's length is even, so they keep to odd slots)
      auto wait_v = [&](int i) {
        if constexpr (MOD != MOD_NONE) return mbar_wait(&v_ok[i % NS], (i / NS) & 1, lim, W_FWD_V_OK);
        return wait_item(i);
      };

      int it = 0;                                  // K/V ring loads consumed
      uint32_t q_par = 0, p_par = 0;               // bit t: parity of the next q_full / p_full phase
      bool ok = true;
      [[maybe_unused]] bool more = true;
      for (int r = 0; ok && (MOD != MOD_NONE ? more : r * G < num_items); ++r) {
        int w;
        if constexpr (MOD == MOD_NONE) {
          w = fwd_item_index(r);
          if (w >= num_items) continue;
        } else if (!take(r, w, ok, more, false)) {
          continue;
        }
        const FwdItem I = fwd_item<CAUSAL, MOD>(p, w);
        if (I.n == 0) continue;
        const int it0 = it;                        // K_j at it0 + 2j, V_j at it0 + 2j + 1
        if (!(ok = wait_item(it0))) break;
#pragma unroll 1
        for (int t = 0; t < 2; ++t) {
          const int ntt = t ? I.n_t1 : I.n_t0;
          if (ntt == 0 || (MOD != MOD_NONE && (t ? I.s_t1 : I.s_t0) > 0)) continue;
          if (!(ok = mbar_wait(&q_full[t], (q_par >> t) & 1u, lim, W_FWD_Q))) break;
          q_par ^= 1u << t;
          tc_fence_after();
          issue_s(t, it0 % NS);
          umma_commit(&s_full[t]);
          if (ntt == 1) umma_commit(&q_empty[t]);
        }
        if (!ok) break;
        umma_commit(&kv_empty[it0 % NS]);
        for (int j = 0; ok && j < I.n; ++j) {
          const int it_v = it0 + 2 * j + 1, it_k = it0 + 2 * j + 2;
          if (!(ok = wait_v(it_v))) break;
          tc_fence_after();
          bool k_ready = false;
#pragma unroll 1
          for (int t = 0; t < 2 && ok; ++t) {
            const int ntt = t ? I.n_t1 : I.n_t0;
            const int st = MOD == MOD_NONE ? 0 : t ? I.s_t1 : I.s_t0;
            if (j >= ntt || j + 1 < st) continue;
            if (j >= st) {
              if (!(ok = mbar_wait(&p_full[t], (p_par >> t) & 1u, lim, W_FWD_P))) break;
              p_par ^= 1u << t;
              tc_fence_after();
              issue_pv(t, it_v % NS, j > st);
            } else {                               // scored: this tile's first step is the next one
              if (!(ok = mbar_wait(&q_full[t], (q_par >> t) & 1u, lim, W_FWD_Q))) break;
              q_par ^= 1u << t;
            }
            if (j + 1 < ntt) {
              if (!k_ready) {
                if (!(ok = wait_item(it_k))) break;
                tc_fence_after();
                k_ready = true;
              }
              issue_s(t, it_k % NS);
              umma_commit(&s_full[t]);
              if (j + 2 == ntt) umma_commit(&q_empty[t]);   // the last S of this Q tile
            } else {
              umma_commit(&o_full[t]);
            }
          }
          if (!ok) break;
          // scored: a step that neither query tile takes part in hands its tiles back all the same
          if (MOD != MOD_NONE && !k_ready && j + 1 < I.n) {
            if (!(ok = wait_item(it_k))) break;
            k_ready = true;
          }
          umma_commit(&kv_empty[it_v % NS]);
          if (k_ready) umma_commit(&kv_empty[it_k % NS]);
        }
        it = it0 + 2 * I.n;
      }
      // nothing may be in flight on the tensor pipe when the CTA tears down
      umma_commit(mma_done);
      mbar_wait(mma_done, 0, lim, W_FWD_DONE);
    }
  } else if (MOD != MOD_NONE && warp == 11) {
    // ------------------------------------------------ V tiles seen in part --
    int it = 0;
    bool ok = true, more = true;
    for (int r = 0; ok && more; ++r) {
      int w;
      if (!take(r, w, ok, more, true)) continue;
      const FwdItem I = fwd_item<CAUSAL, MOD>(p, w);
      int kuni = I.n > 0 ? fwd_key_doc(p, I.b, I.j0) : -1;
      for (int jj = 0; jj < I.n; ++jj) {
        const int j = fwd_tile<MOD>(I, jj), iv = it + 2 * jj + 1, slot = iv % NS;
        const int next = jj + 1 < I.n ? fwd_key_doc(p, I.b, fwd_tile<MOD>(I, jj + 1)) : -1;
        if (!(ok = mbar_wait_warp(&kv_full[slot], (iv / NS) & 1, lim, W_FWD_KV_FULL))) break;
        if ((jj >= I.s_t0 && jj < I.n_t0 && fwd_tile_masked(p, I, 0, j, kuni)) ||
            (jj >= I.s_t1 && jj < I.n_t1 && fwd_tile_masked(p, I, 1, j, kuni)))
          fwd_clean_v<D>(smem + C::KV_OFF + slot * C::TILE_BYTES,
                         reinterpret_cast<uint32_t*>(smem + C::BAD_OFF) + slot * 4);
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_ok[slot]);
        kuni = next;
      }
      it += 2 * I.n;
    }
  }
  // Take the launch budget back only after the softmax warps have returned
  // theirs (named barrier 2): re-acquiring earlier could starve a softmax warp
  // that has not yet grown, and both would wait forever.
  asm volatile("bar.sync 2, %0;" :: "n"(C::THREADS) : "memory");
  setmaxnreg_inc<FWD_LAUNCH_REGS>();
  } else {
    setmaxnreg_inc<FwdRegs<MOD>::SOFTMAX>();
    // ------------------------------------------------------------- softmax --
    const int t = warp >> 2;
    const int wq = warp & 3;                       // TMEM lane quadrant of this warp
    const uint32_t lane_bits = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_s = tmem + lane_bits + t * 128;
    const uint32_t t_o = tmem + lane_bits + 256 + t * D;
    const float sl2 = p.scale_log2;
    int s_cnt = 0, o_cnt = 0;                      // phases consumed on s_full[t], o_full[t]
    [[maybe_unused]] int it = 0;                   // scored: K/V ring entries of the items before
    bool ok = true;
    constexpr bool CAP = (MOD & MOD_CAP) != 0, BIAS = (MOD & MOD_BIAS) != 0, FINE = (MOD & MOD_FINE) != 0;
    // scored: constant pairs (the polynomial's coefficients carry the cap)
    [[maybe_unused]] f2 cscale = 0, ctwo = 0, cy = 0, ck0 = 0, ck1 = 0, ck2 = 0, ck3 = 0, ck4 = 0, ck5 = 0;
    if constexpr (MOD != MOD_NONE && !(MOD & MOD_CAP)) cscale = f2_dup(sl2);
    if constexpr ((MOD & MOD_BIAS) != 0) ctwo = f2_dup(2.f);
    [[maybe_unused]] const float ysc = p.sc.y_scale, cap2 = p.sc.cap_log2, m_base = fmaxf(cap2 - FWD_CAP_ROOM, 0.f);
    if constexpr (CAP) {
      cy = f2_dup(p.sc.y_scale);
      ck0 = f2_dup(FA_TANH_C0 * cap2);
      ck1 = f2_dup(FA_TANH_C1 * cap2);
      ck2 = f2_dup(FA_TANH_C2 * cap2);
      ck3 = f2_dup(FA_TANH_C3 * cap2);
      ck4 = f2_dup(FA_TANH_C4 * cap2);
      ck5 = f2_dup(FA_TANH_C5 * cap2);
    }
    [[maybe_unused]] bool more = true;
    for (int r = 0; ok && (MOD != MOD_NONE ? more : r * G < num_items); ++r) {
      int w;
      if constexpr (MOD == MOD_NONE) {
        w = fwd_item_index(r);
        if (w >= num_items) continue;
      } else if (!take(r, w, ok, more, true)) {
        continue;
      }
      const FwdItem I = fwd_item<CAUSAL, MOD>(p, w);
      if (MOD != MOD_NONE && t == 1 && p.item_rows == 128) { it += 2 * I.n; continue; }
      const int b = I.b, h = I.h;
      const int row_tile0 = I.q0 + t * 128;
      const int row = row_tile0 + wq * 32 + lane;    // global query row of this thread
      const int nt = t ? I.n_t1 : I.n_t0;
      const int st = MOD == MOD_NONE ? 0 : t ? I.s_t1 : I.s_t0;
      // l: exact fp32 sum of p (for LSE); lr: sum of the bf16-rounded p that the
      // P.V product uses (the normaliser of O)
      float m_used = -INFINITY, l = 0.f, lr = 0.f;
      [[maybe_unused]] int qid = -1, kuni = -1;    // scored: this row's document, the next key tile's
      [[maybe_unused]] bool poison = false;        // scored: the row may see a V row holding an inf or NaN
      [[maybe_unused]] float slope2 = 0.f;
      if constexpr (MOD != MOD_NONE) {
        if (p.sc.q_docs != nullptr && nt > 0) {
          if (row < p.Lq) qid = p.sc.q_docs[static_cast<size_t>(b) * p.Lq + row];
          kuni = fwd_key_doc(p, b, fwd_tile<MOD>(I, st));
          // a row without a document sees nothing: any reference does, and the
          // warp is spared the search for one in every tile
          if (qid < 0) m_used = 0.f;
        }
        if constexpr ((MOD & MOD_BIAS) != 0) slope2 = p.sc.slopes[h] * LOG2E;
      }
      [[maybe_unused]] f2 cslope = 0;
      if constexpr ((MOD & MOD_BIAS) != 0) cslope = f2_dup(slope2);

      for (int j = st; j < nt; ++j) {
        [[maybe_unused]] uint32_t m[4];            // scored: the columns this row sees
        [[maybe_unused]] bool masked = false, looked = false;
        if constexpr (MOD != MOD_NONE) {
          const int jt = fwd_tile<MOD>(I, j), kb0 = jt * 128;
          masked = fwd_tile_masked(p, I, t, jt, kuni);
          looked = masked || (j >= (t ? I.s_t0 : I.s_t1) && j < (t ? I.n_t0 : I.n_t1) &&
                              fwd_tile_masked(p, I, t ^ 1, jt, kuni));
#pragma unroll
          for (int w4 = 0; w4 < 4; ++w4) m[w4] = 0xffffffffu;
          if (masked) {
            const int lim_c = p.sc.causal ? min(p.Lk, max(row + off + 1, I.pre)) - kb0 : p.Lk - kb0;
#pragma unroll
            for (int w4 = 0; w4 < 4; ++w4) m[w4] = bits_below(lim_c, w4);
          }
          if (masked && p.sc.q_docs != nullptr) {
            int kid[4];
#pragma unroll
            for (int w4 = 0; w4 < 4; ++w4) {
              const int key = kb0 + w4 * 32 + lane;
              kid[w4] = key < p.Lk ? p.sc.k_docs[static_cast<size_t>(b) * p.Lk + key] : -1;
            }
            doc_bits(qid, kid, m);
          }
          if (j + 1 < nt) kuni = fwd_key_doc(p, b, fwd_tile<MOD>(I, j + 1));
        }
        if (!(ok = mbar_wait_warp(&s_full[t], s_cnt & 1, lim, W_FWD_S))) break;
        ++s_cnt;
        tc_fence_after();
        if constexpr (MOD != MOD_NONE) {
          // which V rows were cleared (V comes along with K, so this is seldom a
          // wait, and the flags need not outlive the scores).  Only after S: the
          // product thread is then past the ring's earlier entries, and the parity
          // names this entry's phase and not the one before the last
          if (looked) {
            const int iv = it + 2 * j + 1;
            if (!(ok = mbar_wait_warp(&v_ok[iv % NS], (iv / NS) & 1, lim, W_FWD_V_OK))) break;
            const uint4 bw = *reinterpret_cast<const uint4*>(smem + C::BAD_OFF + (iv % NS) * 16);
            poison |= ((bw.x & m[0]) | (bw.y & m[1]) | (bw.z & m[2]) | (bw.w & m[3])) != 0u;
          }
        }
        float ls0 = 0.f, ls1 = 0.f, lr0 = 0.f, lr1 = 0.f;
        if constexpr (CAP) {
          // ------------------------------------------------- capped scores --
          // The cap bounds every score, so the reference needs no search: it is
          // cap2 - 24 (at least 0) less the bias of the nearest key seen so far,
          // which keeps p below 2^24 (2^32 with a bias, whose reference follows
          // FWD_TAU behind) and a row's largest p above 2^(24 - 2 cap2), 2^-122 at
          // FWD_CAP_FREE: sums of 2^24 terms p v stay in fp32 for |v| < 2^64.  A
          // larger cap, or a bias that grows with the distance (a negative slope):
          // the tile's largest score is looked for first.  Without a search no tile is exponentiated twice,
          // so S can be read 32 columns at a time and the loop stay rolled: fully
          // unrolled, the polynomial's code outgrows the instruction cache.
          const int kb0 = fwd_tile<MOD>(I, j) * 128, pos = row + off;
          const bool cross = BIAS && (!p.sc.causal || I.pre > 0) && kb0 + 127 > row_tile0 + off;
          float m_want = m_base;
          if constexpr (BIAS) {
            // distance to the nearest key of the tile that this row sees
            int near = max(max(kb0 - pos, pos - (kb0 + 127)), 0);
            if (masked) near = nearest_bit(m, pos - kb0);
            m_want = near < 0 ? -INFINITY : fmaf(-slope2, static_cast<float>(near), m_base);
          }
          if (cap2 > FWD_CAP_FREE || (BIAS && slope2 < 0.f)) {
            m_want = -INFINITY;
  #pragma unroll 1
            for (int qr = 0; qr < 4; ++qr) {
              uint32_t xr[32];
              tmem_ld_32x32b_x32(t_s + qr * 32, xr);
              const uint32_t bits = qr == 0 ? m[0] : qr == 1 ? m[1] : qr == 2 ? m[2] : m[3];
  #pragma unroll
              for (int c = 0; c < 32; ++c) {
                float x = tanh_mufu(__uint_as_float(xr[c]) * ysc) * cap2;
                if constexpr (BIAS) x = fmaf(-slope2, fabsf(static_cast<float>(kb0 + qr * 32 + c - pos)), x);
                m_want = fmaxf(m_want, (bits >> c) & 1u ? x : -INFINITY);
              }
            }
          }
          const bool resc = m_want > m_used + FWD_TAU;                 // false while both are -inf
          float alpha = 1.f;
          if (resc) { alpha = ex2_approx(m_used - m_want); l *= alpha; lr *= alpha; m_used = m_want; }
          if (j > st && __any_sync(0xffffffffu, resc)) {
  #pragma unroll 1
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t ov[32];
              tmem_ld_32x32b_x32(t_o + c0, ov);
  #pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
              tmem_st_32x32b_x32(t_o + c0, ov);
            }
          }
          const float msub = (m_used == -INFINITY) ? 0.f : m_used;
          const f2 nm = f2_pack(-msub, -msub);
          f2 sum = f2_pack(0.f, 0.f), off2 = sum;                      // of p, and of what its two parts leave out
          float d0 = static_cast<float>(kb0 - pos);                    // distance key - query of the chunk's column 0
  #pragma unroll 1
          for (int qr = 0; qr < 4; ++qr) {
            uint32_t xr[32];
            tmem_ld_32x32b_x32(t_s + qr * 32, xr);
            const uint32_t bits = qr == 0 ? m[0] : qr == 1 ? m[1] : qr == 2 ? m[2] : m[3];
            f2 y[16];
            float umax = 0.f;                                          // largest squared tanh argument
  #pragma unroll
            for (int i = 0; i < 16; ++i) {
              y[i] = f2_mul(f2_pack(__uint_as_float(xr[2 * i]), __uint_as_float(xr[2 * i + 1])), cy);
              float u0, u1;
              f2_get(f2_mul(y[i], y[i]), u0, u1);
              umax = fmax3(umax, u0, u1);
            }
            // GEN: with the mask and the bias' absolute value; EXACT: arguments past FA_TANH_LIMIT too
            auto chunk = [&](auto gen_c, auto exact_c) {
              constexpr bool GEN = decltype(gen_c)::value, EXACT = decltype(exact_c)::value;
              uint32_t pk[16], pl[16];
              f2 dist = f2_pack(d0, d0 + 1.f);
  #pragma unroll
              for (int i = 0; i < 16; ++i) {
                f2 x, b = nm;
                if constexpr (BIAS) {
                  f2 d = dist;
                  if constexpr (GEN) {
                    float t0, t1;
                    f2_get(d, t0, t1);
                    d = f2_pack(-fabsf(t0), -fabsf(t1));
                  }
                  b = f2_fma(d, cslope, nm);
                  dist = f2_add(dist, ctwo);
                }
                const f2 u = f2_mul(y[i], y[i]);
                f2 q = f2_fma(u, ck5, ck4);
                q = f2_fma(q, u, ck3);
                q = f2_fma(q, u, ck2);
                q = f2_fma(q, u, ck1);
                q = f2_fma(q, u, ck0);
                x = f2_fma(y[i], q, b);
                if constexpr (EXACT) {                                 // each argument by itself: fa_score.cuh
                  float y0, y1, u0, u1, x0, x1, e0, e1;
                  f2_get(y[i], y0, y1);
                  f2_get(u, u0, u1);
                  f2_get(x, x0, x1);
                  f2_get(f2_fma(f2_pack(tanh_mufu(y0), tanh_mufu(y1)), f2_pack(cap2, cap2), b), e0, e1);
                  constexpr float L2 = FA_TANH_LIMIT * FA_TANH_LIMIT;
                  x = f2_pack(u0 <= L2 ? x0 : e0, u1 <= L2 ? x1 : e1);
                }
                float p0, p1;
                f2_get(x, p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                if constexpr (GEN) {
                  p0 = (bits >> (2 * i)) & 1u ? p0 : 0.f;
                  p1 = (bits >> (2 * i + 1)) & 1u ? p1 : 0.f;
                }
                pk[i] = pack_bf16x2(p0, p1);
                sum = f2_add(sum, f2_pack(p0, p1));
                float r0, r1;
                resid_bf16x2(pk[i], p0, p1, r0, r1);
                pl[i] = pack_bf16x2(r0, r1);
                resid_bf16x2(pl[i], r0, r1, r0, r1);
                off2 = f2_add(off2, f2_pack(r0, r1));
              }
              // over this chunk's own columns of S: 16 of P, then 16 of its second part
              tmem_st_32x32b_x16(t_s + qr * 32, pk);
              tmem_st_32x32b_x16(t_s + qr * 32 + 16, pl);
            };
            if (__any_sync(0xffffffffu, !(umax <= FA_TANH_LIMIT * FA_TANH_LIMIT))) chunk(std::true_type{}, std::true_type{});
            else if (masked || cross) chunk(std::true_type{}, std::false_type{});
            else chunk(std::false_type{}, std::false_type{});
            d0 += 32.f;
          }
          f2_get(sum, ls0, ls1);
          f2_get(off2, lr0, lr1);
          lr0 = ls0 - lr0; lr1 = ls1 - lr1;
        } else {
        uint32_t sr[128];
        tmem_ld_32x32b_x128(t_s, sr);
        float* s = reinterpret_cast<float*>(sr);
        if constexpr (MOD != MOD_NONE) {
          if (masked) {
#pragma unroll
            for (int c = 0; c < 128; ++c) s[c] = ((m[c >> 5] >> (c & 31)) & 1u) ? s[c] : -INFINITY;
          }
          if constexpr (BIAS) {
            // keys after their query (not causal, or in the prefix): the loops below
            // add slope2 * (key - query), which is twice the distance too much there
            if ((!p.sc.causal || I.pre > 0) && fwd_tile<MOD>(I, j) * 128 + 127 > row_tile0 + off) {
              const float fix = -2.f * slope2 / sl2;
              float t0 = static_cast<float>(fwd_tile<MOD>(I, j) * 128 - row - off);
#pragma unroll
              for (int c = 0; c < 128; ++c) {
                s[c] = fmaf(fix, fmaxf(t0, 0.f), s[c]);
                t0 += 1.f;
              }
            }
          }
        }
        [[maybe_unused]] const float d0 = static_cast<float>(fwd_tile<MOD>(I, j) * 128 - row - off);
        const int kbase = j * 128;
        const bool need_mask = MOD != MOD_NONE ? masked : (kbase + 128 > p.Lk) || (CAUSAL && kbase + 127 > row_tile0 + off);
        if (MOD == MOD_NONE && need_mask) {
          int lim_c = p.Lk - kbase;
          if (CAUSAL) lim_c = min(lim_c, row + off + 1 - kbase);
  #pragma unroll
          for (int c = 0; c < 128; ++c) s[c] = (c < lim_c) ? s[c] : -INFINITY;
        }
        // P = 2^(s*scale*log2e - m), packed to bf16 and stored over the first 64
        // columns of S; ls = exact sum, lr = sum of the bf16 values (O's normaliser)
        auto exp_tile = [&](float msub, bool use_poly) {
          ls0 = ls1 = lr0 = lr1 = 0.f;
          if constexpr (FINE) {
            const f2 nm = f2_pack(-msub, -msub);
            f2 sum = f2_pack(0.f, 0.f), off2 = sum;                    // of p, and of what its two parts leave out
            [[maybe_unused]] f2 dist = f2_pack(d0, d0 + 1.f);
  #pragma unroll
            for (int qr = 0; qr < 4; ++qr) {
              uint32_t pk[16], pl[16];
  #pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int c = qr * 32 + 2 * i;
                f2 b = nm;
                if constexpr (BIAS) {
                  b = f2_fma(dist, cslope, nm);
                  dist = f2_add(dist, ctwo);
                }
                float p0, p1;
                f2_get(f2_fma(f2_pack(s[c], s[c + 1]), cscale, b), p0, p1);
                p0 = ex2_approx(p0);
                p1 = ex2_approx(p1);
                pk[i] = pack_bf16x2(p0, p1);
                sum = f2_add(sum, f2_pack(p0, p1));
                float r0, r1;
                resid_bf16x2(pk[i], p0, p1, r0, r1);
                pl[i] = pack_bf16x2(r0, r1);
                resid_bf16x2(pl[i], r0, r1, r0, r1);
                off2 = f2_add(off2, f2_pack(r0, r1));
              }
              tmem_st_32x32b_x16(t_s + qr * 16, pk);
              tmem_st_32x32b_x16(t_s + 64 + qr * 16, pl);
            }
            f2_get(sum, ls0, ls1);
            f2_get(off2, lr0, lr1);
            lr0 = ls0 - lr0; lr1 = ls1 - lr1;
          } else {
  #pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[32];
  #pragma unroll
            for (int i = 0; i < 32; ++i) {
              const int c = half * 64 + 2 * i;
              float x0, x1, p0, p1;
              ffma2(x0, x1, s[c], s[c + 1], sl2, sl2, -msub, -msub);
              if (use_poly && fwd_poly_pair(i)) {
                exp2_poly2(x0, x1, p0, p1);
              } else {
                p0 = ex2_approx(x0);
                p1 = ex2_approx(x1);
              }
              pk[i] = pack_bf16x2(p0, p1);
              fadd2(ls0, ls1, ls0, ls1, p0, p1);
              add_bf16x2_f32(lr0, lr1, pk[i]);
            }
            tmem_st_32x32b_x32(t_s + half * 32, pk);
          }
          }
        };
        if constexpr (FP8) {
          // tile max first, then P = 2^(s - m + FWD_F8_P_LOG2) as e4m3, four per column
          float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
  #pragma unroll
          for (int c = 4; c < 128; c += 4) {
            mx0 = fmaxf(mx0, s[c]); mx1 = fmaxf(mx1, s[c + 1]); mx2 = fmaxf(mx2, s[c + 2]); mx3 = fmaxf(mx3, s[c + 3]);
          }
          const float m_tile = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * sl2;
          const bool resc = m_tile > m_used + FWD_F8_TAU;   // false while both are -inf
          float alpha = 1.f;
          if (resc) { alpha = ex2_approx(m_used - m_tile); l *= alpha; lr *= alpha; m_used = m_tile; }
          if (j > st && __any_sync(0xffffffffu, resc)) {
  #pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t ov[32];
              tmem_ld_32x32b_x32(t_o + c0, ov);
  #pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
              tmem_st_32x32b_x32(t_o + c0, ov);
            }
          }
          const float msub = (m_used == -INFINITY) ? 0.f : m_used - FWD_F8_P_LOG2;
  #pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t pk[16];
  #pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int c = half * 64 + 4 * i;
              float x0, x1, x2, x3;
              ffma2(x0, x1, s[c], s[c + 1], sl2, sl2, -msub, -msub);
              ffma2(x2, x3, s[c + 2], s[c + 3], sl2, sl2, -msub, -msub);
              const float p0 = ex2_approx(x0), p1 = ex2_approx(x1), p2 = ex2_approx(x2), p3 = ex2_approx(x3);
              pk[i] = pack_e4m3x4(p0, p1, p2, p3);
              fadd2(ls0, ls1, ls0, ls1, p0, p1);
              fadd2(ls0, ls1, ls0, ls1, p2, p3);
              add_e4m3x4_f32(lr0, lr1, pk[i]);
            }
            tmem_st_32x32b_x16(t_s + half * 16, pk);
          }
        } else {
        bool slow = __any_sync(0xffffffffu, m_used == -INFINITY);
        [[maybe_unused]] bool over = true;           // this row's own P against its reference is too large, or not known
        if (!slow) {
          // the branch keeps the polynomial loop and the all-MUFU loop apart, so
          // that the compiler cannot evaluate both and select
          if (need_mask) exp_tile(m_used, false);
          else exp_tile(m_used, true);
          over = !(ls0 + ls1 <= FWD_FAST_LIMIT);
          slow = __any_sync(0xffffffffu, over);
        }
        if (slow) {
          float mx0 = s[0], mx1 = s[1], mx2 = s[2], mx3 = s[3];
          if constexpr (BIAS) {
            float t0 = d0;
            mx0 = mx1 = -INFINITY;
  #pragma unroll
            for (int c = 0; c < 128; c += 2) {
              mx0 = fmaxf(mx0, fmaf(s[c], sl2, t0 * slope2));
              mx1 = fmaxf(mx1, fmaf(s[c + 1], sl2, (t0 + 1.f) * slope2));
              t0 += 2.f;
            }
            mx2 = mx3 = mx0;
          } else {
  #pragma unroll
          for (int c = 4; c < 128; c += 4) {
            mx0 = fmaxf(mx0, s[c]); mx1 = fmaxf(mx1, s[c + 1]); mx2 = fmaxf(mx2, s[c + 2]); mx3 = fmaxf(mx3, s[c + 3]);
          }
          }
          const float m_tile = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3)) * (BIAS ? 1.f : sl2);
          // scored: a row that could have kept its reference keeps it, whatever the
          // warp's other rows ran into
          const bool resc = m_tile > m_used + FWD_TAU && (MOD == MOD_NONE || over);   // false while both are -inf
          float alpha = 1.f;
          if (resc) { alpha = ex2_approx(m_used - m_tile); l *= alpha; lr *= alpha; m_used = m_tile; }
          if (j > st && __any_sync(0xffffffffu, resc)) {
  #pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) {
              uint32_t ov[32];
              tmem_ld_32x32b_x32(t_o + c0, ov);
  #pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
              tmem_st_32x32b_x32(t_o + c0, ov);
            }
          }
          exp_tile((m_used == -INFINITY) ? 0.f : m_used, false);
        }
        }
        }
        l += ls0 + ls1;
        lr += lr0 + lr1;
        // a row of NaN scores has no maximum; any reference does, and the warp's
        // other rows keep to their own
        if (MOD != MOD_NONE && l != l && m_used == -INFINITY) m_used = 0.f;
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&p_full[t]);
      }
      it += 2 * I.n;

      // ------------------------------------------------------------ epilogue --
      const bool have_o = ok && nt > 0 && mbar_wait_warp(&o_full[t], o_cnt & 1, lim, W_FWD_O);
      if (nt > 0) ++o_cnt;
      if (have_o) tc_fence_after();
      const bool has = MOD != MOD_NONE ? l != 0.f : l > 0.f;   // scored: a NaN sum gives a NaN LSE
      float inv_l = (lr > 0.f) ? p.o_scale / lr : 0.f;
      if constexpr (MOD != MOD_NONE) {
        if (poison || lr != lr) inv_l = __int_as_float(0x7fffffff);
      }
      const float m_lse = FP8 ? m_used - FWD_F8_P_LOG2 : m_used;   // the reference l is counted against
      if (row < p.Lq && p.lse != nullptr) {
        const size_t li = (static_cast<size_t>(b) * p.Hq + h) * p.Lq + row;
        if (index_ok(li, 1, static_cast<size_t>(p.B) * p.Hq * p.Lq, W_IDX_FWD_LSE))
          p.lse[li] = has ? (m_lse + log2f(l)) * LN2 : -INFINITY;
      }
      const size_t orow = (static_cast<size_t>(b) * p.Lq + row) * p.Hq + h;
#pragma unroll
      for (int c0 = 0; c0 < D; c0 += 32) {
        uint32_t ov[32];
        if (have_o) {
          tmem_ld_32x32b_x32(t_o + c0, ov);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) ov[i] = 0u;
        }
        if (row >= p.Lq) continue;
        if (!index_ok(orow * D + c0, 32, static_cast<size_t>(p.B) * p.Lq * p.Hq * D, W_IDX_FWD_O)) continue;
        if (p.o_fp32) {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.o) + orow * D + c0);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(__uint_as_float(ov[4 * i]) * inv_l, __uint_as_float(ov[4 * i + 1]) * inv_l,
                                 __uint_as_float(ov[4 * i + 2]) * inv_l, __uint_as_float(ov[4 * i + 3]) * inv_l);
        } else {
          uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.o) + orow * D + c0);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 wv;
            wv.x = pack_bf16x2(__uint_as_float(ov[8 * i + 0]) * inv_l, __uint_as_float(ov[8 * i + 1]) * inv_l);
            wv.y = pack_bf16x2(__uint_as_float(ov[8 * i + 2]) * inv_l, __uint_as_float(ov[8 * i + 3]) * inv_l);
            wv.z = pack_bf16x2(__uint_as_float(ov[8 * i + 4]) * inv_l, __uint_as_float(ov[8 * i + 5]) * inv_l);
            wv.w = pack_bf16x2(__uint_as_float(ov[8 * i + 6]) * inv_l, __uint_as_float(ov[8 * i + 7]) * inv_l);
            dst[i] = wv;
            if (FINE && p.o_lo != nullptr) {
              const uint32_t hi[4] = {wv.x, wv.y, wv.z, wv.w};
              uint32_t lo[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float r0, r1;
                resid_bf16x2(hi[e], __uint_as_float(ov[8 * i + 2 * e]) * inv_l,
                             __uint_as_float(ov[8 * i + 2 * e + 1]) * inv_l, r0, r1);
                lo[e] = pack_bf16x2(r0, r1);
              }
              reinterpret_cast<uint4*>(p.o_lo + orow * D + c0)[i] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            }
          }
        }
      }
    }
    setmaxnreg_dec<FWD_LAUNCH_REGS>();    // give the extra registers back first
    asm volatile("bar.arrive 2, %0;" :: "n"(C::THREADS) : "memory");
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 10) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace fa
