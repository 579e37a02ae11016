// Eviction from a KV cache by accumulated attention weight: of the n rows of a
// sequence, every kv head keeps its last `recent` ones and, of those before
// them, the keep - recent with the largest weights (equal weights: the lower
// row first; a NaN weight ranks below every number).  The kept rows move, in
// order, to rows 0 .. keep - 1 of the destination, which may be the cache
// itself; sequences of at most `keep` rows are kept whole.
//
//   evict_select_kernel  one block per (sequence, kv head): the threshold
//       weight by radix selection (histograms of 11, 11 and 10 bits of the
//       order-preserving integer image of the fp32 weights), then one pass that
//       writes the kept row numbers in order and the kept weights.  The images
//       of the first EVICT_CACHED rows stay in shared memory, so that the weights
//       are read once; a longer sequence's rest is read again from L2.
//   evict_move_kernel    K or V of one (sequence, kv head).  Into another cache,
//       one block per run of rows.  In place, one block per slice of the row's
//       bytes, in steps of rows, each step read whole before it is written: the
//       kept rows only move down (row r comes from kept[r] >= r), so a step's
//       writes (rows below its end) never touch what a later step reads (rows at
//       or past its end).
//
// It has to read the weights once and to read and write the kept rows.  16
// sequences of 8192 to 32768 rows, 8 heads of 128, 4096 kept: 29 us to select (a
// block per head leaves 20 of 148 SMs idle, and each of the three histograms
// waits for its atomics) and 87 us to move 0.54 GB, the copy rate for pieces of
// 256 bytes (82 us).  One prompt of 4001 rows, 1024 kept: 7 and 4 us, latency.
#pragma once
#include "sm100.cuh"

namespace fa {

// Rows of a sequence: contiguous [B, cap, Hkv, D], or pages [num_pages,
// page_size, Hkv, D] through table [B, pages_per_seq].
struct KvRows {
  uint16_t* k;
  uint16_t* v;
  const int* table;        // nullptr: contiguous
  int cap;                 // rows a sequence can hold
  int page_size, pages_per_seq, num_pages;
};
struct EvictParams {
  KvRows src, dst;
  const float* w_src;      // [B, Hkv, w_src_ld]
  float* w_dst;            // [B, Hkv, w_dst_ld], may be w_src
  const int* len_src;      // [B]
  int* len_dst;            // [B], may be len_src
  int* kept;               // [B, Hkv, keep]: source rows, -1 past the kept ones
  int B, Hkv, D, keep, recent, w_src_ld, w_dst_ld;
  int slice_chunks;        // 16-byte chunks of a row that one move block takes (a power of two)
  int cached;              // rows whose keys the select kernel keeps in shared memory
};

enum : uint32_t { W_EVICT_PAGE = 0x601, W_IDX_EVICT = 0x409 };

// Larger weight, larger key; -0 and +0 alike, NaN below everything.
__device__ __forceinline__ uint32_t evict_key(float w) {
  if (w != w) return 0u;
  const uint32_t b = __float_as_uint(w + 0.f);
  return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr int EVICT_THREADS = 1024;
constexpr int EVICT_BINS = 2048;
constexpr int EVICT_CACHED = 32768;              // 128 KB of keys

__global__ void __launch_bounds__(EVICT_THREADS) evict_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t keys[];             // p.cached of them
  __shared__ int hist[EVICT_BINS];
  __shared__ int warp_sum[32];
  __shared__ int s_bin, s_above;
  const int bh = blockIdx.x, b = bh / p.Hkv, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = max(0, min(p.len_src[b], p.src.cap));
  const float* w = p.w_src + static_cast<size_t>(bh) * p.w_src_ld;
  float* w2 = p.w_dst + static_cast<size_t>(bh) * p.w_dst_ld;
  int* kept = p.kept + static_cast<size_t>(bh) * p.keep;
  const int keep = p.keep;
  if (n <= keep) {
    for (int r = tid; r < keep; r += EVICT_THREADS) {
      kept[r] = r < n ? r : -1;
      if (r < n && w2 != w) w2[r] = w[r];
    }
    return;
  }
  const int need = keep - p.recent, old = n - p.recent;

  // threshold: the need-th largest key of [0, old), most significant bits first
  uint32_t prefix = 0, mask = 0;
  int above = 0;                                  // keys known to lie above the prefix's range
  if (need > 0) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
      hist[tid] = 0;
      hist[tid + EVICT_THREADS] = 0;
      __syncthreads();
      if (pass == 0) {
        for (int i0 = tid; i0 < old; i0 += 8 * EVICT_THREADS) {
          float v[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) v[u] = i0 + u * EVICT_THREADS < old ? w[i0 + u * EVICT_THREADS] : 0.f;
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const int i = i0 + u * EVICT_THREADS;
            if (i >= old) break;
            const uint32_t key = evict_key(v[u]);
            if (i < p.cached) keys[i] = key;
            atomicAdd(&hist[key >> 21], 1);
          }
        }
      } else {
#pragma unroll 4
        for (int i = tid; i < old; i += EVICT_THREADS) {
          const uint32_t key = i < p.cached ? keys[i] : evict_key(w[i]);
          if ((key & mask) == prefix) atomicAdd(&hist[(key >> shift) & (bins - 1)], 1);
        }
      }
      __syncthreads();
      // the bin, from the top, in which the count passes `need`: each thread
      // owns two bins (in descending order), block-wide prefix sums over them
      const int hi = bins - 1 - 2 * tid;
      const int c0 = hi >= 0 ? hist[hi] : 0, c1 = hi >= 1 ? hist[hi - 1] : 0;
      int incl = c0 + c1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      {
        const int v = lane < warp ? warp_sum[lane] : 0;      // the warps before this one
        incl += __reduce_add_sync(0xffffffffu, v) + above;
      }
      const int excl = incl - c0 - c1;
      if (excl < need && excl + c0 >= need) { s_bin = hi; s_above = excl; }
      else if (excl + c0 < need && incl >= need) { s_bin = hi - 1; s_above = excl + c0; }
      __syncthreads();
      prefix |= static_cast<uint32_t>(s_bin) << shift;
      mask |= static_cast<uint32_t>(bins - 1) << shift;
      above = s_above;
    }
  }
  const int ties = need - above;                  // rows at the threshold that are kept: the lowest ones

  // Kept rows in order: sweeps of 4096 rows, 128 per warp, ties and picks counted
  // by ballots.  In place a sweep's weights are all read before it writes any
  // (the first barrier), and it writes at most up to where it has read.
  constexpr int U = 4;
  int pos = 0, tied = 0;                          // kept so far, rows at the threshold so far
  float ahead[U];                                 // the next sweep's weights, on their way
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int i = (warp * U + u) * 32 + lane;
    ahead[u] = i < n ? w[i] : 0.f;
  }
  for (int i0 = 0; i0 < n; i0 += U * EVICT_THREADS) {
    float wi[U];
    uint32_t eqs[U], gts[U];
    int n_eq = 0, n_gt = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + (U * 32 + warp * U + u) * 32 + lane;
      wi[u] = ahead[u];
      ahead[u] = i < n ? w[i] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + (warp * U + u) * 32 + lane;
      const uint32_t key = evict_key(wi[u]);
      eqs[u] = __ballot_sync(0xffffffffu, need > 0 && i < old && key == prefix);
      gts[u] = __ballot_sync(0xffffffffu, (need > 0 && i < old && key > prefix) || (i >= old && i < n));
      n_eq += __popc(eqs[u]);
      n_gt += __popc(gts[u]);
    }
    if (lane == 0) warp_sum[warp] = n_eq | (n_gt << 16);
    __syncthreads();
    // both counts of the warps before this one, and of all (each at most 4096)
    const int v = warp_sum[lane];
    const int all = __reduce_add_sync(0xffffffffu, v), before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    int eq_at = before & 0xffff, gt_at = before >> 16;   // of this sweep, before this warp's next 32 rows
    const int room = max(ties - tied, 0);                // ties still to keep when the sweep starts
    const uint32_t lower = (1u << lane) - 1u;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int my_eq = eq_at + __popc(eqs[u] & lower), my_gt = gt_at + __popc(gts[u] & lower);
      const bool pick = ((gts[u] >> lane) & 1u) || (((eqs[u] >> lane) & 1u) && my_eq < room);
      const int at = pos + my_gt + min(room, my_eq);
      if (pick && index_ok(at, 1, keep, W_IDX_EVICT)) {
        kept[at] = i0 + (warp * U + u) * 32 + lane;
        w2[at] = wi[u];
      }
      eq_at += __popc(eqs[u]);
      gt_at += __popc(gts[u]);
    }
    pos += (all >> 16) + min(room, all & 0xffff);
    tied += all & 0xffff;
    __syncthreads();
  }
}

// Element offset of row r of sequence b (kv head 0), or -1 for a page outside the pool.
__device__ __forceinline__ long long evict_row(const KvRows& s, int b, int r, int Hkv, int D) {
  if (s.table == nullptr) return (static_cast<long long>(b) * s.cap + r) * Hkv * D;
  const int pg = s.table[static_cast<size_t>(b) * s.pages_per_seq + r / s.page_size];
  if (pg < 0 || pg >= s.num_pages) return -1;
  return (static_cast<long long>(pg) * s.page_size + r % s.page_size) * Hkv * D;
}

constexpr int EVICT_MOVE_THREADS = 256;
constexpr int EVICT_UNROLL = 8;                   // 16-byte chunks a thread holds per step

template <bool IN_PLACE>
__global__ void __launch_bounds__(EVICT_MOVE_THREADS) evict_move_kernel(const EvictParams p) {
  const int b = blockIdx.z, hkv = blockIdx.y / 2, which = blockIdx.y & 1;
  const int bh = b * p.Hkv + hkv;
  const uint16_t* src = which ? p.src.v : p.src.k;
  uint16_t* dst = which ? p.dst.v : p.dst.k;
  const int* kept = p.kept + static_cast<size_t>(bh) * p.keep;
  const int cps = p.slice_chunks, rows_per = EVICT_MOVE_THREADS / cps, step = rows_per * EVICT_UNROLL;
  // a block owns a slice of the columns and, into another cache, a run of rows
  const int slices = (p.D / 8 + cps - 1) / cps;
  const int slice = IN_PLACE ? blockIdx.x : blockIdx.x % slices;
  const int first = IN_PLACE ? 0 : static_cast<int>(blockIdx.x) / slices * step;
  const int last = IN_PLACE ? p.keep : min(p.keep, first + step);
  const int col = (slice * cps + threadIdx.x % cps) * 8;         // first element of this thread's chunk
  const int r_in = threadIdx.x / cps;
  const bool col_ok = col < p.D;
  pdl_wait();                                                    // the row numbers are written
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0)
    p.len_dst[b] = min(max(0, min(p.len_src[b], p.src.cap)), p.keep);
  for (int r0 = first; r0 < last; r0 += step) {
    uint4 val[EVICT_UNROLL];
    int from[EVICT_UNROLL];
    bool any = false;
#pragma unroll
    for (int u = 0; u < EVICT_UNROLL; ++u) {
      const int r = r0 + u * rows_per + r_in;
      from[u] = col_ok && r < p.keep ? kept[r] : -1;
      if (IN_PLACE && from[u] == r) from[u] = -1;                // already in its place
      any |= from[u] >= 0;
    }
    // a step without any row to move: the first rows of a cache in place
    if (IN_PLACE && !__syncthreads_or(any)) continue;
#pragma unroll
    for (int u = 0; u < EVICT_UNROLL; ++u) {
      if (from[u] < 0) continue;
      const long long at = evict_row(p.src, b, from[u], p.Hkv, p.D);
      if (at < 0) { record_status(FA_DEV_BAD_INPUT, W_EVICT_PAGE); from[u] = -1; continue; }
      val[u] = *reinterpret_cast<const uint4*>(src + at + hkv * p.D + col);
    }
    if (IN_PLACE) __syncthreads();                               // the step is read before any of it is written
#pragma unroll
    for (int u = 0; u < EVICT_UNROLL; ++u) {
      if (from[u] < 0) continue;
      const int r = r0 + u * rows_per + r_in;
      const long long at = evict_row(p.dst, b, r, p.Hkv, p.D);
      if (at < 0) { record_status(FA_DEV_BAD_INPUT, W_EVICT_PAGE); continue; }
      const size_t pool = (p.dst.table ? static_cast<size_t>(p.dst.num_pages) * p.dst.page_size
                                       : static_cast<size_t>(p.B) * p.dst.cap) * p.Hkv * p.D;
      if (!index_ok(static_cast<size_t>(at) + hkv * p.D + col, 8, pool, W_IDX_EVICT)) continue;
      *reinterpret_cast<uint4*>(dst + at + hkv * p.D + col) = val[u];
    }
  }
}

}  // namespace fa
