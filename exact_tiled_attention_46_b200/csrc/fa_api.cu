// Host side of the C ABI declared in include/fa.h: argument checks, tensor-map
// encoding, kernel selection and launches.  Nothing here allocates device
// memory or synchronises (except fa_device_status, which says so).
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <algorithm>
#include <mutex>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"
#include "sm100.cuh"
#include "fa_fwd.cuh"
#include "fa_decode.cuh"
#include "fa_bwd.cuh"
#include "fa_weights.cuh"
#include "fa_evict.cuh"

namespace {

constexpr int kAbiVersion = 1;
constexpr int kDecodeChunk = 1024;
std::atomic<unsigned long long> g_wait_limit_ns{2000000000ull};

// ---------------------------------------------------------- tensor maps ----
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(ptr);
  });
  return fn;
}

// 4-D map over a [B, L, H, D] tensor (bf16; fp32 or single bytes when asked):
// dims (D, H, L, B), box (box_d, 1, box_rows, 1).
bool map_bshd(CUtensorMap* m, const void* base, int B, int L, int H, int D, int box_d, int box_rows, bool sw128,
              bool fp32 = false, bool bytes = false) {
  EncodeTiledFn enc = encode_fn();
  if (enc == nullptr) return false;
  const cuuint64_t es_bytes = fp32 ? 4 : bytes ? 1 : 2;
  cuuint64_t dims[4] = {cuuint64_t(D), cuuint64_t(H), cuuint64_t(L), cuuint64_t(B)};
  cuuint64_t strides[3] = {cuuint64_t(D) * es_bytes, cuuint64_t(H) * D * es_bytes, cuuint64_t(L) * H * D * es_bytes};
  cuuint32_t box[4] = {cuuint32_t(box_d), 1, cuuint32_t(box_rows), 1};
  cuuint32_t es[4] = {1, 1, 1, 1};
  const CUtensorMapDataType dt = fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  return enc(m, dt, 4, const_cast<void*>(base),
             dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, sw128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// ------------------------------------------------------------- helpers -----
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool scale_ok(float s) { return std::isfinite(s) && s > 0.f; }
bool fits_int(long long x) { return x >= 0 && x <= INT_MAX; }

// Sets the dynamic shared-memory limit of `func` once per device.
template <typename F>
bool ensure_smem_attr(F* func, int bytes, std::atomic<uint64_t>& done_mask) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
  const uint64_t bit = uint64_t(1) << dev;
  if (done_mask.load(std::memory_order_acquire) & bit) return true;
  if (cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return false;
  done_mask.fetch_or(bit, std::memory_order_acq_rel);
  return true;
}

fa_status launch_status() { return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA; }

// Launches `kernel` so that it may start while its predecessor in the stream
// still runs (it waits for it with pdl_wait before it reads anything).
template <typename... P>
fa_status launch_after(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t st, const P&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Number of SMs of the current device (cached per device); 0 on failure.
int sm_count() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 0;
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

__global__ void fill_empty_rows_kernel(void* o, float* lse, size_t n_o, size_t n_lse, int o_fp32) {
  const size_t i = blockIdx.x * size_t(blockDim.x) + threadIdx.x;
  const size_t stride = size_t(gridDim.x) * blockDim.x;
  for (size_t k = i; k < n_o; k += stride) {
    if (o_fp32) static_cast<float*>(o)[k] = 0.f;
    else static_cast<uint16_t*>(o)[k] = 0;
  }
  if (lse != nullptr)
    for (size_t k = i; k < n_lse; k += stride) lse[k] = -INFINITY;
}

__global__ void selftest_wait_kernel(unsigned long long limit_ns) {
  __shared__ uint64_t bar;
  if (threadIdx.x == 0) { fa::mbar_init(&bar, 1); fa::fence_mbar_init(); }
  __syncthreads();
  fa::mbar_wait(&bar, 0, limit_ns, 0x9001);   // no thread ever arrives
}

__global__ void selftest_exp2_poly_kernel(const float* x, float* y, int n) {
  const int i = 2 * (blockIdx.x * blockDim.x + threadIdx.x);
  if (i + 1 < n) {
    fa::exp2_poly2(x[i], x[i + 1], y[i], y[i + 1]);
  } else if (i < n) {
    float unused;
    fa::exp2_poly2(x[i], x[i], y[i], unused);
  }
}

// The forward and backward kernels move registers between warpgroups
// (setmaxnreg); that is only safe when the launch allocation per thread is
// exactly the one the split was computed for.  A build that allocates
// differently is refused, never run.  The result is kept per kernel
// instantiation (each launch_* template instance owns its `state`), because
// all instantiations of one kernel template share a function type.
enum : int { REGS_UNKNOWN = 0, REGS_MATCH = 1, REGS_MISMATCH = 2 };
template <typename F>
bool launch_regs_match(F* func, int expected, std::atomic<int>& state) {
  int s = state.load();
  if (s == REGS_UNKNOWN) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, func) != cudaSuccess) return false;
    s = (a.numRegs == expected) ? REGS_MATCH : REGS_MISMATCH;
    state.store(s);
  }
  return s == REGS_MATCH;
}
// Per-instantiation guard states, indexed by kernel_slot().  The scored variants
// (mod odd: MOD_SCORED with or without cap and bias) follow the plain ones.
std::atomic<int> g_regs_state[34];
constexpr int kernel_slot(bool bwd, int D, bool causal, bool fp8 = false, int mod = fa::MOD_NONE) {
  if (mod != fa::MOD_NONE) return 10 + (bwd ? 16 : 0) + (D == 128 ? (bwd ? 4 : 8) : 0) + (mod >> 1);
  return fp8 ? 8 + (causal ? 1 : 0) : (bwd ? 4 : 0) + (D == 128 ? 2 : 0) + (causal ? 1 : 0);
}

template <int D, bool CAUSAL, bool FP8 = false, int MOD = fa::MOD_NONE>
fa_status launch_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const fa::FwdParams& p,
                     long long grid, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  constexpr int smem = fa::FwdCfg<D, FP8, MOD>::SMEM_BYTES;
  if (!launch_regs_match(fa::fwd_kernel<D, CAUSAL, FP8, MOD>, fa::FWD_LAUNCH_REGS,
                         g_regs_state[kernel_slot(false, D, CAUSAL, FP8, MOD)]))
    return FA_ERR_UNSUPPORTED;
  if (!ensure_smem_attr(fa::fwd_kernel<D, CAUSAL, FP8, MOD>, smem, attr_done)) return FA_ERR_CUDA;
  if constexpr (MOD != fa::MOD_NONE)
    return launch_after(fa::fwd_kernel<D, CAUSAL, FP8, MOD>, dim3(static_cast<unsigned>(grid)),
                        dim3(fa::FwdCfg<D, FP8, MOD>::THREADS), smem, st, mq, mk, mv, p);
  fa::fwd_kernel<D, CAUSAL, FP8, MOD>
      <<<static_cast<unsigned>(grid), fa::FwdCfg<D, FP8, MOD>::THREADS, smem, st>>>(mq, mk, mv, p);
  return launch_status();
}

template <int D, int GP, bool PAGED, bool APPEND, bool SCORED = false>
fa_status launch_decode(const CUtensorMap& mk, const CUtensorMap& mv, const fa::DecParams& p, unsigned grid,
                        cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  using C = fa::DecCfg<D, GP>;
  if (!ensure_smem_attr(fa::decode_split_kernel<D, GP, PAGED, APPEND, SCORED>, C::SMEM_BYTES, attr_done))
    return FA_ERR_CUDA;
  fa::decode_split_kernel<D, GP, PAGED, APPEND, SCORED><<<grid, C::THREADS, C::SMEM_BYTES, st>>>(mk, mv, p);
  return launch_status();
}

template <bool PAGED, bool APPEND>
fa_status dispatch_decode(int D, int GP, const CUtensorMap& mk, const CUtensorMap& mv, const fa::DecParams& p,
                          unsigned grid, cudaStream_t st) {
  if (D == 128)
    return GP == 4 ? launch_decode<128, 4, PAGED, APPEND>(mk, mv, p, grid, st)
         : GP == 2 ? launch_decode<128, 2, PAGED, APPEND>(mk, mv, p, grid, st)
                   : launch_decode<128, 1, PAGED, APPEND>(mk, mv, p, grid, st);
  return GP == 4 ? launch_decode<64, 4, PAGED, APPEND>(mk, mv, p, grid, st)
       : GP == 2 ? launch_decode<64, 2, PAGED, APPEND>(mk, mv, p, grid, st)
                 : launch_decode<64, 1, PAGED, APPEND>(mk, mv, p, grid, st);
}

template <bool PAGED, bool APPEND>
fa_status dispatch_decode_scored(int D, int GP, const CUtensorMap& mk, const CUtensorMap& mv, const fa::DecParams& p,
                                 unsigned grid, cudaStream_t st) {
  if (D == 128)
    return GP == 8 ? launch_decode<128, 8, PAGED, APPEND, true>(mk, mv, p, grid, st)
         : GP == 4 ? launch_decode<128, 4, PAGED, APPEND, true>(mk, mv, p, grid, st)
                   : launch_decode<128, 1, PAGED, APPEND, true>(mk, mv, p, grid, st);
  return GP == 8 ? launch_decode<64, 8, PAGED, APPEND, true>(mk, mv, p, grid, st)
       : GP == 4 ? launch_decode<64, 4, PAGED, APPEND, true>(mk, mv, p, grid, st)
                 : launch_decode<64, 1, PAGED, APPEND, true>(mk, mv, p, grid, st);
}

// One split-KV decode call, every variant: cache rows from a contiguous cache
// (page_table == nullptr: "pages" are the sequences, page_size = Lmax) or a
// page pool, and, when k_new != nullptr, the new token's rows attended and
// appended.  Checks every argument before anything is launched.
fa_status run_decode(const void* q, const void* k_new, const void* v_new, const void* k_cache, const void* v_cache,
                     const int* page_table, const int* seqlens, void* o, float* lse, int B, int Hq, int Hkv,
                     int num_pages, int page_size, int pages_per_seq, int D, float scale, int o_dtype,
                     void* workspace, size_t workspace_bytes, cudaStream_t st) {
  const bool paged = page_table != nullptr, append = k_new != nullptr || v_new != nullptr;
  if (!q || !k_cache || !v_cache || !seqlens || !o || !workspace) return FA_ERR_INVALID_ARG;
  if (append && (!k_new || !v_new)) return FA_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (num_pages <= 0 || page_size <= 0 || pages_per_seq <= 0) return FA_ERR_INVALID_ARG;
  if (paged && page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
  if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_BF16 && o_dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned256(workspace) ||
      !aligned16(k_new) || !aligned16(v_new))
    return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(seqlens) & 3u) != 0 || (reinterpret_cast<uintptr_t>(lse) & 3u) != 0 ||
      (reinterpret_cast<uintptr_t>(page_table) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  const long long cap = static_cast<long long>(page_size) * pages_per_seq;
  if (cap + 1 > INT_MAX) return FA_ERR_UNSUPPORTED;
  const int G = Hq / Hkv;
  const int GP = (G % 4 == 0) ? 4 : (G % 2 == 0) ? 2 : 1;
  const int HG = Hkv * (G / GP);
  const long long keys = cap + (append ? 1 : 0);
  const long long max_splits = (keys + kDecodeChunk - 1) / kDecodeChunk;
  if (!fits_int(static_cast<long long>(B) * max_splits * HG) || !fits_int(static_cast<long long>(B) * Hq))
    return FA_ERR_UNSUPPORTED;
  if (workspace_bytes < fa_decode_workspace_size(B, Hq, static_cast<int>(keys), D)) return FA_ERR_INVALID_ARG;
  const int sub_rows = (page_size % 32 == 0 || !paged) ? 32 : 16;
  CUtensorMap mk, mv;
  // boxes of 64 dimensions (128 bytes, 128-byte swizzle) by sub_rows rows
  if (!map_bshd(&mk, k_cache, num_pages, page_size, Hkv, D, 64, sub_rows, true) ||
      !map_bshd(&mv, v_cache, num_pages, page_size, Hkv, D, 64, sub_rows, true))
    return FA_ERR_CUDA;
  float* o_part = static_cast<float*>(workspace);
  const size_t lse_off = align_up(size_t(B) * Hq * max_splits * D * 4, 256);
  float* lse_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + lse_off);
  int* counter = reinterpret_cast<int*>(static_cast<char*>(workspace) + lse_off +
                                        align_up(size_t(B) * Hq * max_splits * 4, 256));
  if (cudaMemsetAsync(counter, 0, sizeof(int), st) != cudaSuccess) return FA_ERR_CUDA;
  fa::DecParams p;
  p.seqlens = seqlens; p.q = static_cast<const uint16_t*>(q);
  p.k_new = static_cast<const uint16_t*>(k_new); p.v_new = static_cast<const uint16_t*>(v_new);
  p.k_cache = static_cast<uint16_t*>(const_cast<void*>(k_cache));
  p.v_cache = static_cast<uint16_t*>(const_cast<void*>(v_cache));
  p.page_table = page_table;
  p.o_part = o_part; p.lse_part = lse_part; p.work_counter = counter;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.max_splits = static_cast<int>(max_splits); p.chunk = kDecodeChunk;
  p.cap = static_cast<int>(cap); p.page_size = page_size; p.pages_per_seq = pages_per_seq; p.num_pages = num_pages;
  p.sub_rows = sub_rows;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_limit_ns = g_wait_limit_ns.load();
  // persistent grid: as many CTAs as fit (3 per SM), never more than there can be items
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  const long long items = static_cast<long long>(B) * max_splits * HG;
  const unsigned grid = static_cast<unsigned>(std::min<long long>(items, 3LL * sms));
  fa_status s;
  if (paged) s = append ? dispatch_decode<true, true>(D, GP, mk, mv, p, grid, st)
                        : dispatch_decode<true, false>(D, GP, mk, mv, p, grid, st);
  else s = append ? dispatch_decode<false, true>(D, GP, mk, mv, p, grid, st)
                  : dispatch_decode<false, false>(D, GP, mk, mv, p, grid, st);
  if (s != FA_OK) return s;
  fa::CombineParams c;
  c.o_part = o_part; c.lse_part = lse_part; c.counts = seqlens; c.o = o; c.lse = lse;
  c.B = B; c.Hq = Hq; c.D = D; c.max_splits = static_cast<int>(max_splits); c.chunk = kDecodeChunk;
  c.o_fp32 = (o_dtype == FA_FP32); c.cap = static_cast<int>(cap); c.append = append ? 1 : 0;
  fa::decode_combine_kernel<<<B * Hq, 128, 0, st>>>(c);
  return launch_status();
}

template <int D, bool CAUSAL, int MOD = fa::MOD_NONE>
fa_status launch_bwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const CUtensorMap& mdo,
                     const CUtensorMap& mdq, const fa::BwdParams& p, unsigned grid, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  constexpr int smem = fa::BwdCfg<D>::SMEM_BYTES;
  if (!launch_regs_match(fa::bwd_main_kernel<D, CAUSAL, MOD>, fa::BWD_LAUNCH_REGS,
                         g_regs_state[kernel_slot(true, D, CAUSAL, false, MOD)]))
    return FA_ERR_UNSUPPORTED;
  if (!ensure_smem_attr(fa::bwd_main_kernel<D, CAUSAL, MOD>, smem, attr_done)) return FA_ERR_CUDA;
  if constexpr (MOD != fa::MOD_NONE)
    return launch_after(fa::bwd_main_kernel<D, CAUSAL, MOD>, dim3(grid), dim3(fa::BwdCfg<D>::THREADS), smem, st, mq, mk,
                        mv, mdo, mdq, p);
  fa::bwd_main_kernel<D, CAUSAL, MOD><<<grid, fa::BwdCfg<D>::THREADS, smem, st>>>(mq, mk, mv, mdo, mdq, p);
  return launch_status();
}

// ------------------------------------------------------- scored attention --
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
cudaStream_t st_of(fa_stream_t s) { return reinterpret_cast<cudaStream_t>(s); }
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}
bool cap_ok(float c) { return std::isfinite(c) && c >= 0.f; }

// Checks a fa_score and fills the kernels' parameters; *mod gets the variant.
fa_status score_params(const fa_score* s, float scale, int causal, int Lq, int Lk, fa::ScoreParams* sp, int* mod) {
  if (s == nullptr || !cap_ok(s->softcap)) return FA_ERR_INVALID_ARG;
  if (!aligned4(s->slopes) || !aligned4(s->q_docs) || !aligned4(s->k_docs) || !aligned4(s->prefix))
    return FA_ERR_INVALID_ARG;
  if (Lq > 0 && Lk > 0 && (s->q_docs == nullptr) != (s->k_docs == nullptr)) return FA_ERR_INVALID_ARG;
  if (s->prefix != nullptr && !causal) return FA_ERR_INVALID_ARG;
  if (s->slopes != nullptr && (Lq >= (1 << 24) || Lk >= (1 << 24))) return FA_ERR_UNSUPPORTED;
  if (s->slopes != nullptr && scale < 0x1p-64f) return FA_ERR_UNSUPPORTED;   // slope / scale must stay finite
  const float y = s->softcap > 0.f ? scale / s->softcap : 0.f;
  if (!std::isfinite(y) || !std::isfinite(s->softcap * fa::LOG2E)) return FA_ERR_INVALID_ARG;
  sp->y_scale = y;
  sp->cap_log2 = s->softcap * fa::LOG2E;
  sp->slopes = s->slopes;
  sp->q_docs = s->q_docs;
  sp->k_docs = s->k_docs;
  sp->prefix = s->prefix;
  sp->q_meta = sp->k_meta = nullptr;
  sp->counter = nullptr;
  sp->causal = causal != 0;
  *mod = fa::MOD_SCORED | (s->softcap > 0.f ? fa::MOD_CAP : 0) | (s->slopes != nullptr ? fa::MOD_BIAS : 0);
  return FA_OK;
}

// The tile facts of the documents, into `ws` (fa_scored_workspace_size bytes).
fa_status launch_meta(fa::ScoreParams* sp, int B, int Lq, int Lk, void* ws, cudaStream_t st,
                      uint32_t* zero8 = nullptr, uint32_t* unseen = nullptr) {
  if (sp->q_docs == nullptr) return FA_OK;
  const int nq = (Lq + 127) / 128, nk = (Lk + 127) / 128;
  int4* q_meta = static_cast<int4*>(ws);
  int4* k_meta = q_meta + size_t(B) * nq;
  sp->counter = reinterpret_cast<int*>(k_meta + size_t(B) * nk);
  fa::score_meta_kernel<<<dim3(nq + nk, B), 256, 0, st>>>(sp->q_docs, sp->k_docs, Lq, Lk, q_meta, k_meta, sp->counter,
                                                            zero8, unseen, sp->causal, sp->prefix);
  sp->q_meta = q_meta;
  sp->k_meta = k_meta;
  return launch_status();
}

// Calls f with the variant as a constant.
template <typename F>
fa_status with_mod(int mod, F f) {
  switch (mod) {
    case fa::MOD_SCORED: return f(std::integral_constant<int, fa::MOD_SCORED>{});
    case fa::MOD_SCORED | fa::MOD_CAP: return f(std::integral_constant<int, fa::MOD_SCORED | fa::MOD_CAP>{});
    case fa::MOD_SCORED | fa::MOD_BIAS: return f(std::integral_constant<int, fa::MOD_SCORED | fa::MOD_BIAS>{});
    default:
      return f(std::integral_constant<int, fa::MOD_SCORED | fa::MOD_CAP | fa::MOD_BIAS>{});
  }
}

// Query rows per item of the scored forward: two query tiles share an item's
// keys and overlap each other's products and exponentials; a grid that would not
// fill the SMs takes one.
int fwd_item_rows(int B, int Hq, int Lq, int sms) {
  return ((static_cast<long long>(Lq) + 255) / 256) * B * Hq < sms ? 128 : 256;
}
// (Query range, batch row, head) items of the scored forward.
long long fwd_items(int B, int Hq, int Lq, int rows) {
  return (static_cast<long long>(Lq) + rows - 1) / rows * B * Hq;
}

// The scored forward's launch, arguments checked and the documents' tile facts
// in `sp`; `fine` asks for P in two parts even where nothing is changed.
fa_status run_fwd_scored(const void* q, const void* k, const void* v, void* o, void* o_lo, float* lse, int B, int Hq,
                         int Hkv, int Lq, int Lk, int D, float scale, const fa::ScoreParams& sp, int mod, bool fine,
                         int o_dtype, int sms, cudaStream_t st) {
  CUtensorMap mq, mk, mv;
  if (!map_bshd(&mq, q, B, Lq, Hq, D, 64, 128, true) || !map_bshd(&mk, k, B, Lk, Hkv, D, 64, 128, true) ||
      !map_bshd(&mv, v, B, Lk, Hkv, D, 64, 128, true))
    return FA_ERR_CUDA;
  fa::FwdParams p;
  p.sc = sp;
  p.item_rows = fwd_item_rows(B, Hq, Lq, sms);
  const long long items = fwd_items(B, Hq, Lq, p.item_rows);
  if (items <= sms) p.sc.counter = nullptr;       // one item per CTA: nothing to deal out
  p.o = o; p.lse = lse; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Lq = Lq; p.Lk = Lk;
  p.o_lo = static_cast<uint16_t*>(o_lo);
  p.num_pairs = (Lq + p.item_rows - 1) / p.item_rows;
  p.scale_log2 = scale * fa::LOG2E;
  p.o_scale = 1.f;
  p.o_fp32 = (o_dtype == FA_FP32);
  p.wait_limit_ns = g_wait_limit_ns.load();
  const long long grid = items < sms ? items : sms;
  // nothing changed and no rounding asked for: plain attention, fa_fwd_ex's bits
  if (mod == fa::MOD_SCORED && sp.q_docs == nullptr && sp.prefix == nullptr && !fine)
    return D == 128 ? launch_fwd<128, true, false, fa::MOD_SCORED>(mq, mk, mv, p, grid, st)
                    : launch_fwd<64, true, false, fa::MOD_SCORED>(mq, mk, mv, p, grid, st);
  return with_mod(mod, [&](auto m) {
    constexpr int FINE = decltype(m)::value | fa::MOD_FINE;
    return D == 128 ? launch_fwd<128, true, false, FINE>(mq, mk, mv, p, grid, st)
                    : launch_fwd<64, true, false, FINE>(mq, mk, mv, p, grid, st);
  });
}

// Parts into which fa_key_weights cuts the (query tile, head) pairs of a key
// tile: enough items for six rounds of the SMs, which even out the causal
// tiles' work, but no part shorter than eight pairs (two per warpgroup).  Parts
// cost a reduction launch and their sums' traffic (a causal prompt of 4095
// tokens, 32 query and 8 kv heads: 126 us for two rounds, 105 us for six).
int key_weight_parts(int B, int Hq, int Hkv, int Lq, int Lk, int sms) {
  const long long tiles = ((long long)Lk + 127) / 128 * B * Hkv;
  const long long pairs = ((long long)Lq + 127) / 128 * (Hq / Hkv);
  long long parts = (6LL * sms + tiles - 1) / std::max<long long>(tiles, 1);
  parts = std::min(parts, (pairs + 7) / 8);
  return static_cast<int>(std::max<long long>(1, std::min<long long>(parts, 64)));
}
constexpr int kMaxSms = 148;   // workspace sizes do not depend on the current device

template <int D, int MOD>
fa_status launch_kw(const CUtensorMap& mq, const CUtensorMap& mk, const fa::KwParams& p, unsigned grid,
                    cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  using C = fa::KwCfg<D>;
  if (!ensure_smem_attr(fa::kw_kernel<D, MOD>, C::SMEM_BYTES, attr_done)) return FA_ERR_CUDA;
  return launch_after(fa::kw_kernel<D, MOD>, dim3(grid), dim3(C::THREADS), C::SMEM_BYTES, st, mq, mk, p);
}

// Keys per chunk of a scored decode: the longest of 1024, 512, 256, 128 that
// still gives every SM two rounds of its three CTAs when the cache is full.
int scored_chunk(int B, int Hq, int Hkv, int rows) {
  const int G = Hq / Hkv;
  const long long groups = static_cast<long long>(B) * Hkv * ((G + 7) / 8);
  for (int chunk = 1024; chunk > 128; chunk /= 2)
    if (groups * ((static_cast<long long>(rows) + chunk - 1) / chunk) >= 6LL * kMaxSms) return chunk;
  return 128;
}

// Scratch of fa_decode_splitkv_static: the split-KV partial results of the
// most recent call.  In host code this name is only a stand-in for the device
// array; its device address is looked up per device with cudaGetSymbolAddress.
static __device__ __align__(256) unsigned char g_decode_static_scratch[FA_DECODE_STATIC_SCRATCH_BYTES];
std::mutex g_static_mu;
void* g_static_scratch_ptr[64] = {};

// One backward call, plain (score == nullptr) or scored.
fa_status run_bwd(const void* q, const void* k, const void* v, const void* o, const void* o_lo, const void* dO,
                  const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Lq, int Lk, int D, float scale, int causal,
                  const fa_score* score, int grad_dtype, void* workspace, size_t workspace_bytes, cudaStream_t st) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Lq < 0 || Lk < 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  // empty tensors may come with null pointers
  if (Lq > 0 && (!q || !o || !dO || !lse || !dq)) return FA_ERR_INVALID_ARG;
  if (Lk > 0 && (!k || !v || !dk || !dv)) return FA_ERR_INVALID_ARG;
  if (Lq > 0 && Lk > 0 && !workspace) return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
  if (grad_dtype != FA_BF16 && grad_dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(dO) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned256(workspace) || (reinterpret_cast<uintptr_t>(lse) & 3u))
    return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  fa::ScoreParams sp{};
  int mod = fa::MOD_NONE;
  if (score != nullptr) {
    const fa_status s = score_params(score, scale, causal, Lq, Lk, &sp, &mod);
    if (s != FA_OK) return s;
    if (B > 65535 || !fits_int(fwd_items(B, Hq, Lq, 128))) return FA_ERR_UNSUPPORTED;
  }
  if (workspace_bytes < (score ? fa_bwd_scored_workspace_size(B, Hq, Lq, Lk, D) : fa_bwd_workspace_size(B, Hq, Lq, D)))
    return FA_ERR_INVALID_ARG;
  if (!fits_int(static_cast<long long>((Lk + 127) / 128) * B * Hkv)) return FA_ERR_UNSUPPORTED;
  const int sms = sm_count();
  const size_t g_elt = grad_dtype == FA_FP32 ? 4 : 2;
  if (Lq == 0 || Lk == 0) {   // no (query, key) pair: the gradients that exist are zero
    const size_t nk = size_t(B) * Lk * Hkv * D * g_elt, nq = size_t(B) * Lq * Hq * D * g_elt;
    if ((nk && (cudaMemsetAsync(dk, 0, nk, st) != cudaSuccess || cudaMemsetAsync(dv, 0, nk, st) != cudaSuccess)) ||
        (nq && cudaMemsetAsync(dq, 0, nq, st) != cudaSuccess))
      return FA_ERR_CUDA;
    return FA_OK;
  }
  const int lq_pad = static_cast<int>(align_up(size_t(Lq), 128));
  const size_t acc_bytes = size_t(B) * Lq * Hq * D * 4;
  const size_t row_bytes = align_up(size_t(B) * Hq * lq_pad * 4, 256);
  const size_t h_bytes = align_up(size_t(B) * Lq * Hq * D * 2, 256);
  char* ws = static_cast<char*>(workspace);
  float* dq_acc = reinterpret_cast<float*>(ws);
  float* lse2 = reinterpret_cast<float*>(ws + align_up(acc_bytes, 256));
  float* delta = reinterpret_cast<float*>(reinterpret_cast<char*>(lse2) + row_bytes);
  uint16_t* q16 = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(delta) + row_bytes);
  uint16_t* do16 = reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(q16) + h_bytes);
  uint32_t* amax = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(do16) + h_bytes);
  int* counter = reinterpret_cast<int*>(amax + 4);                 // the main kernel's work counter
  const uint16_t *q_in = static_cast<const uint16_t*>(q), *k_in = static_cast<const uint16_t*>(k);
  const uint16_t *v_in = static_cast<const uint16_t*>(v), *do_in = static_cast<const uint16_t*>(dO);
  const size_t nq = size_t(B) * Lq * Hq * D, nk = size_t(B) * Lk * Hkv * D;
  const unsigned amax_blocks = static_cast<unsigned>(std::min<size_t>((std::max(nq, nk) / 8 + 1023) / 1024, 148 * 4));
  const size_t chunks = size_t(B) * lq_pad * Hq * (D / 8);         // one thread per 16-byte chunk of a row
  const unsigned pre_blocks = static_cast<unsigned>(std::min<size_t>((chunks + 255) / 256, 148 * 16));
  uint32_t* unseen = nullptr;                                      // keys that no query sees, with documents
  if (score == nullptr) {
    if (cudaMemsetAsync(dq_acc, 0, acc_bytes, st) != cudaSuccess || cudaMemsetAsync(amax, 0, 32, st) != cudaSuccess)
      return FA_ERR_CUDA;
    fa::bwd_amax_kernel<false><<<dim3(amax_blocks, 4), 256, 0, st>>>(q_in, k_in, v_in, do_in, nq, nk, amax);
    if (launch_status() != FA_OK) return FA_ERR_CUDA;
    fa::bwd_pre_kernel<false><<<pre_blocks, 256, 0, st>>>(static_cast<const uint16_t*>(o), nullptr, nullptr, do_in, q_in,
                                                          lse, amax, lse2, delta, q16, do16, B, Hq, Lq, lq_pad, D,
                                                          nullptr);
    if (launch_status() != FA_OK) return FA_ERR_CUDA;
  } else {
    // a chain of kernels that start while their predecessor ends; the first one
    // zeroes the maxima and the work counter, bwd_pre_kernel the dQ accumulator
    fa_status s;
    if (sp.k_docs != nullptr) unseen = reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(amax) + 256 + fa_scored_workspace_size(B, Lq, Lk));
    if (sp.k_docs == nullptr) {
      if (cudaMemsetAsync(amax, 0, 32, st) != cudaSuccess) return FA_ERR_CUDA;
    } else if ((s = launch_meta(&sp, B, Lq, Lk, reinterpret_cast<char*>(amax) + 256, st, amax, unseen)) !=
               FA_OK) {
      return s;
    }
    // without what rounding took off o, O is formed again, in two bf16 parts that
    // lie where bwd_pre_kernel puts q16 and do16 (each chunk is read by the thread
    // that then writes it): 83 us of 537 for the training step B2 Hq16 Hkv4 L2048 D128 with a cap
    const uint16_t *lo = static_cast<const uint16_t*>(o_lo), *o_new = nullptr;
    if (lo == nullptr) {
      if (sms <= 0) return FA_ERR_CUDA;
      s = run_fwd_scored(q, k, v, q16, do16, nullptr, B, Hq, Hkv, Lq, Lk, D, scale, sp, mod, true, FA_BF16, sms, st);
      if (s != FA_OK) return s;
      o_new = q16;
      lo = do16;
    }
    // every row counts unless documents, or more queries than keys under the
    // causal mask, leave some without a key
    if (sp.k_docs != nullptr || (causal && Lq > Lk)) {
      const size_t units = size_t(B) * ((std::max(Lq, Lk) + 31) / 32);
      s = launch_after(fa::bwd_amax_scored_kernel, dim3(static_cast<unsigned>(std::min<size_t>(units, 148 * 4)), 4),
                       dim3(256), 0, st, q_in, k_in, v_in, do_in, amax, lse,
                       static_cast<const uint32_t*>(unseen), B, Hq, Hkv, Lq, Lk, D);
    } else {
      s = launch_after(fa::bwd_amax_kernel<true>, dim3(amax_blocks, 4), dim3(256), 0, st, q_in, k_in, v_in, do_in, nq, nk,
                       amax);
    }
    if (s != FA_OK) return s;
    s = launch_after(fa::bwd_pre_kernel<true>, dim3(pre_blocks), dim3(256), 0, st, static_cast<const uint16_t*>(o), o_new,
                     lo, do_in, q_in, lse, static_cast<const uint32_t*>(amax), lse2, delta,
                     q16, do16, B, Hq, Lq, lq_pad, D, dq_acc);
    if (s != FA_OK) return s;
  }
  CUtensorMap mq, mk, mv, mdo, mdq;
  // q and dO are read from their fp16 copies (2-byte elements: the bf16 map
  // type only sets the element size here), k and v as given; the fp32 dQ
  // accumulator takes reductions of 32-row x 32-column boxes
  if (!map_bshd(&mq, q16, B, Lq, Hq, D, 64, 128, true) || !map_bshd(&mk, k, B, Lk, Hkv, D, 64, 128, true) ||
      !map_bshd(&mv, v, B, Lk, Hkv, D, 64, 128, true) || !map_bshd(&mdo, do16, B, Lq, Hq, D, 64, 128, true) ||
      !map_bshd(&mdq, dq_acc, B, Lq, Hq, D, 32, 32, true, true))
    return FA_ERR_CUDA;
  fa::BwdParams p;
  p.lse2 = lse2; p.delta = delta; p.amax = amax; p.dk = dk; p.dv = dv;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Lq = Lq; p.Lk = Lk; p.Lq_pad = lq_pad;
  p.scale = scale; p.scale_log2 = scale * 1.4426950408889634f; p.g_fp32 = (grad_dtype == FA_FP32);
  p.wait_limit_ns = g_wait_limit_ns.load();
  // persistent: at most one CTA per SM, taking key tiles from the counter
  p.num_items = static_cast<int>(((Lk + 127) / 128) * B * Hkv);
  p.work_counter = counter;
  p.sc = sp;
  p.unseen = unseen;
  if (sms <= 0) return FA_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(std::min(p.num_items, sms));
  fa_status s;
  if (D == 64 && mod == (fa::MOD_SCORED | fa::MOD_CAP) && score->softcap > fa::BWD_MUFU_CAP) mod |= fa::MOD_BIAS;
  if (score != nullptr)
    s = with_mod(mod, [&](auto m) {
      return D == 128 ? launch_bwd<128, true, decltype(m)::value>(mq, mk, mv, mdo, mdq, p, grid, st)
                      : launch_bwd<64, true, decltype(m)::value>(mq, mk, mv, mdo, mdq, p, grid, st);
    });
  else if (D == 128) s = causal ? launch_bwd<128, true>(mq, mk, mv, mdo, mdq, p, grid, st) : launch_bwd<128, false>(mq, mk, mv, mdo, mdq, p, grid, st);
  else s = causal ? launch_bwd<64, true>(mq, mk, mv, mdo, mdq, p, grid, st) : launch_bwd<64, false>(mq, mk, mv, mdo, mdq, p, grid, st);
  if (s != FA_OK) return s;
  const size_t n = nq;
  const unsigned blocks = static_cast<unsigned>(std::min<size_t>((n / 4 + 255) / 256, 148 * 16));
  if (score != nullptr)
    return launch_after(fa::bwd_post_kernel, dim3(blocks), dim3(256), 0, st, static_cast<const float*>(dq_acc), dq, n, scale,
                        static_cast<const uint32_t*>(amax), D, static_cast<int>(grad_dtype == FA_FP32));
  fa::bwd_post_kernel<<<blocks, 256, 0, st>>>(dq_acc, dq, n, scale, amax, D, grad_dtype == FA_FP32);
  return launch_status();
}

}  // namespace

extern "C" {

int fa_abi_version(void) { return kAbiVersion; }

int fa_debug_build(void) {
#ifdef FA_DEBUG
  return 1;
#else
  return 0;
#endif
}

const char* fa_status_string(int s) {
  switch (s) {
    case FA_OK: return "ok";
    case FA_ERR_INVALID_ARG: return "invalid argument";
    case FA_ERR_UNSUPPORTED: return "unsupported configuration";
    case FA_ERR_CUDA: return "CUDA call failed";
    case FA_ERR_TIMEOUT: return "kernel wait timed out";
    case FA_ERR_DEVICE_INDEX: return "device index check failed (debug build)";
    default: return "unknown status";
  }
}

void fa_set_wait_limit_ns(unsigned long long ns) { g_wait_limit_ns.store(ns > 0 ? ns : 1); }

fa_status fa_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv,
                    int Lq, int Lk, int D, float scale, int causal, int o_dtype, fa_stream_t stream) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Lq < 0 || Lk < 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  // empty tensors may come with null pointers: q/o only matter when Lq > 0, k/v when Lk > 0
  if (Lq > 0 && (!q || !o)) return FA_ERR_INVALID_ARG;
  if (Lq > 0 && Lk > 0 && (!k || !v)) return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_BF16 && o_dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  const long long pairs = (static_cast<long long>(Lq) + 255) / 256;
  const long long items = pairs * B * Hq;          // work items of the persistent grid
  if (!fits_int(items) || !fits_int(static_cast<long long>(B) * Hq)) return FA_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (Lq == 0) return FA_OK;
  if (Lk == 0) {
    const size_t n_o = size_t(B) * Lq * Hq * D, n_l = size_t(B) * Hq * Lq;
    fill_empty_rows_kernel<<<296, 256, 0, st>>>(o, lse, n_o, n_l, o_dtype == FA_FP32);
    return launch_status();
  }
  CUtensorMap mq, mk, mv;
  if (!map_bshd(&mq, q, B, Lq, Hq, D, 64, 128, true) || !map_bshd(&mk, k, B, Lk, Hkv, D, 64, 128, true) ||
      !map_bshd(&mv, v, B, Lk, Hkv, D, 64, 128, true))
    return FA_ERR_CUDA;
  fa::FwdParams p;
  p.o = o; p.lse = lse; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Lq = Lq; p.Lk = Lk;
  p.num_pairs = static_cast<int>(pairs);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.o_scale = 1.f;
  p.o_fp32 = (o_dtype == FA_FP32);
  p.wait_limit_ns = g_wait_limit_ns.load();
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  const long long grid = items < sms ? items : sms;
  if (D == 128) return causal ? launch_fwd<128, true>(mq, mk, mv, p, grid, st) : launch_fwd<128, false>(mq, mk, mv, p, grid, st);
  return causal ? launch_fwd<64, true>(mq, mk, mv, p, grid, st) : launch_fwd<64, false>(mq, mk, mv, p, grid, st);
}

fa_status fa_fwd_fp8(const void* q, const void* k, const void* v, float q_scale, float k_scale, float v_scale,
                     void* o, float* lse, int B, int Hq, int Hkv, int Lq, int Lk, int D, float scale, int causal,
                     int o_dtype, fa_stream_t stream) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Lq < 0 || Lk < 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (Lq > 0 && (!q || !o)) return FA_ERR_INVALID_ARG;
  if (Lq > 0 && Lk > 0 && (!k || !v)) return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale) || !scale_ok(q_scale) || !scale_ok(k_scale) || !scale_ok(v_scale)) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_BF16 && o_dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o)) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(lse) & 3u) != 0) return FA_ERR_INVALID_ARG;
  if (D != 128) return FA_ERR_UNSUPPORTED;
  const long long pairs = (static_cast<long long>(Lq) + 255) / 256;
  const long long items = pairs * B * Hq;
  if (!fits_int(items) || !fits_int(static_cast<long long>(B) * Hq)) return FA_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (Lq == 0) return FA_OK;
  if (Lk == 0) {
    const size_t n_o = size_t(B) * Lq * Hq * D, n_l = size_t(B) * Hq * Lq;
    fill_empty_rows_kernel<<<296, 256, 0, st>>>(o, lse, n_o, n_l, o_dtype == FA_FP32);
    return launch_status();
  }
  CUtensorMap mq, mk, mv;
  if (!map_bshd(&mq, q, B, Lq, Hq, D, 128, 128, true, false, true) ||
      !map_bshd(&mk, k, B, Lk, Hkv, D, 128, 128, true, false, true) ||
      !map_bshd(&mv, v, B, Lk, Hkv, D, 128, 128, true, false, true))
    return FA_ERR_CUDA;
  fa::FwdParams p;
  p.o = o; p.lse = lse; p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Lq = Lq; p.Lk = Lk;
  p.num_pairs = static_cast<int>(pairs);
  p.scale_log2 = scale * q_scale * k_scale * 1.4426950408889634f;
  p.o_scale = v_scale;
  p.o_fp32 = (o_dtype == FA_FP32);
  p.wait_limit_ns = g_wait_limit_ns.load();
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  const long long grid = items < sms ? items : sms;
  return causal ? launch_fwd<128, true, true>(mq, mk, mv, p, grid, st)
                : launch_fwd<128, false, true>(mq, mk, mv, p, grid, st);
}

fa_status fa_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int Hq, int Hkv, int Lq,
                 int Lk, int D, float scale, int causal, fa_stream_t stream) {
  return fa_fwd_ex(q, k, v, o, lse, B, Hq, Hkv, Lq, Lk, D, scale, causal, FA_BF16, stream);
}

int fa_decode_chunk(void) { return kDecodeChunk; }

size_t fa_decode_workspace_size(int B, int Hq, int Lmax, int D) {
  if (B <= 0 || Hq <= 0 || Lmax < 0 || D <= 0) return 0;
  const size_t ms = std::max<size_t>(1, (size_t(Lmax) + kDecodeChunk - 1) / kDecodeChunk);
  // partial outputs, partial LSEs, the work counter of the split kernel
  return align_up(size_t(B) * Hq * ms * D * 4, 256) + align_up(size_t(B) * Hq * ms * 4, 256) + 256;
}

fa_status fa_decode_combine(const float* o_part, const float* lse_part, const int* num_splits, void* o, float* lse,
                            int B, int Hq, int D, int max_splits, int o_dtype, fa_stream_t stream) {
  if (!o_part || !lse_part || !o) return FA_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || D <= 0 || D > 4096 || max_splits <= 0) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_BF16 && o_dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!fits_int(static_cast<long long>(B) * Hq)) return FA_ERR_UNSUPPORTED;
  fa::CombineParams c;
  c.o_part = o_part; c.lse_part = lse_part; c.counts = num_splits; c.o = o; c.lse = lse;
  c.B = B; c.Hq = Hq; c.D = D; c.max_splits = max_splits; c.chunk = 0; c.o_fp32 = (o_dtype == FA_FP32);
  c.cap = 0; c.append = 0;
  fa::decode_combine_kernel<<<B * Hq, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(c);
  return launch_status();
}

fa_status fa_decode_splitkv(const void* q, const void* k_cache, const void* v_cache, const int* seqlens, void* o,
                            float* lse, int B, int Hq, int Hkv, int Lmax, int D, float scale, int o_dtype,
                            void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (B <= 0 || Lmax <= 0) return FA_ERR_INVALID_ARG;
  return run_decode(q, nullptr, nullptr, k_cache, v_cache, nullptr, seqlens, o, lse, B, Hq, Hkv, B, Lmax, 1, D,
                    scale, o_dtype, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_decode_append_splitkv(const void* q, const void* k_new, const void* v_new, void* k_cache,
                                   void* v_cache, const int* seqlens, void* o, float* lse, int B, int Hq, int Hkv,
                                   int Lmax, int D, float scale, int o_dtype, void* workspace,
                                   size_t workspace_bytes, fa_stream_t stream) {
  if (B <= 0 || Lmax <= 0 || !k_new || !v_new) return FA_ERR_INVALID_ARG;
  return run_decode(q, k_new, v_new, k_cache, v_cache, nullptr, seqlens, o, lse, B, Hq, Hkv, B, Lmax, 1, D, scale,
                    o_dtype, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_decode_paged_splitkv(const void* q, const void* k_new, const void* v_new, void* k_pages,
                                  void* v_pages, const int* page_table, const int* seqlens, void* o, float* lse,
                                  int B, int Hq, int Hkv, int num_pages, int page_size, int pages_per_seq, int D,
                                  float scale, int o_dtype, void* workspace, size_t workspace_bytes,
                                  fa_stream_t stream) {
  if (!page_table) return FA_ERR_INVALID_ARG;
  return run_decode(q, k_new, v_new, k_pages, v_pages, page_table, seqlens, o, lse, B, Hq, Hkv, num_pages,
                    page_size, pages_per_seq, D, scale, o_dtype, workspace, workspace_bytes,
                    reinterpret_cast<cudaStream_t>(stream));
}

fa_status fa_attn_merge(const float* o_a, const float* lse_a, const float* o_b, const float* lse_b, void* o_out,
                        float* lse_out, int B, int H, int L, int D, int o_dtype, fa_stream_t stream) {
  if (B <= 0 || H <= 0 || L < 0 || D <= 0 || D % 4 != 0) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_BF16 && o_dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (L == 0) return FA_OK;
  if (!o_a || !lse_a || !o_b || !lse_b || !o_out) return FA_ERR_INVALID_ARG;
  if (!aligned16(o_a) || !aligned16(o_b) || !aligned16(o_out)) return FA_ERR_INVALID_ARG;
  if (((reinterpret_cast<uintptr_t>(lse_a) | reinterpret_cast<uintptr_t>(lse_b) |
        reinterpret_cast<uintptr_t>(lse_out)) & 3u) != 0)
    return FA_ERR_INVALID_ARG;
  // the output may be either input: every element is read by the thread that writes it, before it writes
  fa::MergeParams p;
  p.o_a = o_a; p.lse_a = lse_a; p.o_b = o_b; p.lse_b = lse_b; p.o_out = o_out; p.lse_out = lse_out;
  p.B = B; p.H = H; p.L = L; p.D = D; p.o_fp32 = (o_dtype == FA_FP32);
  const size_t rows = size_t(B) * L * H;
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  const unsigned blocks = static_cast<unsigned>(std::min<size_t>((rows + 7) / 8, size_t(sms) * 16));
  fa::attn_merge_kernel<<<blocks, 256, 0, reinterpret_cast<cudaStream_t>(stream)>>>(p);
  return launch_status();
}

fa_status fa_decode_splitkv_static(const void* q, const void* k_cache, const void* v_cache, const int* seqlens,
                                   void* o, float* lse, int B, int Hq, int Hkv, int Lmax, int D, float scale,
                                   int o_dtype, fa_stream_t stream) {
  if (fa_decode_workspace_size(B, Hq, Lmax, D) > FA_DECODE_STATIC_SCRATCH_BYTES) return FA_ERR_UNSUPPORTED;
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FA_ERR_CUDA;
  void* scratch = nullptr;
  {
    // set-up, once per device, with that device current
    std::lock_guard<std::mutex> lock(g_static_mu);
    if (g_static_scratch_ptr[dev] == nullptr) {
      void* ptr = nullptr;
      if (cudaGetSymbolAddress(&ptr, g_decode_static_scratch) != cudaSuccess || ptr == nullptr) return FA_ERR_CUDA;
      g_static_scratch_ptr[dev] = ptr;
    }
    scratch = g_static_scratch_ptr[dev];
  }
  return fa_decode_splitkv(q, k_cache, v_cache, seqlens, o, lse, B, Hq, Hkv, Lmax, D, scale, o_dtype, scratch,
                           FA_DECODE_STATIC_SCRATCH_BYTES, stream);
}

size_t fa_bwd_workspace_size(int B, int Hq, int Lq, int D) {
  if (B <= 0 || Hq <= 0 || Lq < 0 || D <= 0) return 0;
  const size_t lq_pad = align_up(size_t(Lq), 128);
  // fp32 dQ accumulator, the padded log2 LSE and Delta rows, the scaled fp16
  // copies of q and dO, the four input maxima
  return align_up(size_t(B) * Lq * Hq * D * 4, 256) + 2 * align_up(size_t(B) * Hq * lq_pad * 4, 256) +
         2 * align_up(size_t(B) * Lq * Hq * D * 2, 256) + 256;
}

fa_status fa_bwd(const void* q, const void* k, const void* v, const void* o, const void* dO, const float* lse,
                 void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Lq, int Lk, int D, float scale, int causal,
                 int grad_dtype, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  return run_bwd(q, k, v, o, nullptr, dO, lse, dq, dk, dv, B, Hq, Hkv, Lq, Lk, D, scale, causal, nullptr, grad_dtype, workspace,
                 workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t fa_scored_workspace_size(int B, int Lq, int Lk) {
  if (B <= 0 || Lq < 0 || Lk < 0) return 0;
  return align_up(size_t(B) * (size_t(Lq) / 128 + size_t(Lk) / 128 + 2) * sizeof(int4) + sizeof(int), 256);
}

fa_status fa_fwd_scored(const void* q, const void* k, const void* v, void* o, void* o_lo, float* lse, int B, int Hq, int Hkv,
                        int Lq, int Lk, int D, float scale, int causal, const fa_score* score, int o_dtype,
                        void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Lq < 0 || Lk < 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (Lq > 0 && (!q || !o)) return FA_ERR_INVALID_ARG;
  if (Lq > 0 && Lk > 0 && (!k || !v)) return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale)) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_BF16 && o_dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(o_lo) || !aligned16(workspace) ||
      !aligned4(lse))
    return FA_ERR_INVALID_ARG;
  if (o_lo != nullptr && o_dtype != FA_BF16) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  fa::ScoreParams sp{};
  int mod = fa::MOD_NONE;
  fa_status s = score_params(score, scale, causal, Lq, Lk, &sp, &mod);
  if (s != FA_OK) return s;
  const int sms = sm_count();
  if (!fits_int(fwd_items(B, Hq, Lq, fwd_item_rows(B, Hq, Lq, sms))) || !fits_int(static_cast<long long>(B) * Hq) ||
      B > 65535)
    return FA_ERR_UNSUPPORTED;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (Lq == 0) return FA_OK;
  if (Lk == 0) {
    const size_t n_o = size_t(B) * Lq * Hq * D, n_l = size_t(B) * Hq * Lq;
    fill_empty_rows_kernel<<<296, 256, 0, st>>>(o, lse, n_o, n_l, o_dtype == FA_FP32);
    if (o_lo != nullptr) fill_empty_rows_kernel<<<296, 256, 0, st>>>(o_lo, nullptr, n_o, 0, 0);
    return launch_status();
  }
  if (sp.q_docs != nullptr && (!workspace || workspace_bytes < fa_scored_workspace_size(B, Lq, Lk)))
    return FA_ERR_INVALID_ARG;
  if (sms <= 0) return FA_ERR_CUDA;
  if ((s = launch_meta(&sp, B, Lq, Lk, workspace, st)) != FA_OK) return s;
  return run_fwd_scored(q, k, v, o, o_lo, lse, B, Hq, Hkv, Lq, Lk, D, scale, sp, mod, o_lo != nullptr, o_dtype, sms, st);
}

size_t fa_bwd_scored_workspace_size(int B, int Hq, int Lq, int Lk, int D) {
  if (B <= 0 || Hq <= 0 || Lq < 0 || Lk < 0 || D <= 0) return 0;
  return fa_bwd_workspace_size(B, Hq, Lq, D) + fa_scored_workspace_size(B, Lq, Lk) +
         align_up(size_t(B) * ((size_t(Lk) + 127) / 128) * 16, 256);
}

fa_status fa_bwd_scored(const void* q, const void* k, const void* v, const void* o, const void* o_lo, const void* dO,
                        const float* lse, void* dq, void* dk, void* dv, int B, int Hq, int Hkv, int Lq, int Lk, int D, float scale,
                        int causal, const fa_score* score, int grad_dtype, void* workspace, size_t workspace_bytes,
                        fa_stream_t stream) {
  if (score == nullptr) return FA_ERR_INVALID_ARG;
  if (!aligned16(o_lo)) return FA_ERR_INVALID_ARG;
  return run_bwd(q, k, v, o, o_lo, dO, lse, dq, dk, dv, B, Hq, Hkv, Lq, Lk, D, scale, causal, score, grad_dtype, workspace,
                 workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

size_t fa_decode_scored_workspace_size(int B, int Hq, int Hkv, int rows, int D, int with_weights) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || rows < 0 || D <= 0) return 0;
  const int chunk = scored_chunk(B, Hq, Hkv, rows);
  const size_t ms = std::max<size_t>(1, (size_t(rows) + chunk - 1) / chunk);
  // partial outputs, partial log-sums, the work counter, the scores
  return align_up(size_t(B) * Hq * ms * D * 4, 256) + align_up(size_t(B) * Hq * ms * 4, 256) + 256 +
         (with_weights ? size_t(B) * Hq * align_up(size_t(rows), 4) * 4 : 0);
}

fa_status fa_decode_scored_splitkv(const void* q, const void* k_new, const void* v_new, void* k_cache, void* v_cache,
                                   const int* page_table, const int* seqlens, const int* starts, void* o, float* lse,
                                   float* weights, int weights_ld, int B, int Hq, int Hkv, int num_pages,
                                   int page_size, int pages_per_seq, int D, float scale, float softcap,
                                   const float* slopes, int o_dtype, void* workspace, size_t workspace_bytes,
                                   fa_stream_t stream) {
  const bool paged = page_table != nullptr, append = k_new != nullptr || v_new != nullptr;
  if (!q || !k_cache || !v_cache || !seqlens || !o || !workspace) return FA_ERR_INVALID_ARG;
  if (append && (!k_new || !v_new)) return FA_ERR_INVALID_ARG;
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (num_pages <= 0 || page_size <= 0 || pages_per_seq <= 0) return FA_ERR_INVALID_ARG;
  if (!paged && (num_pages != B || pages_per_seq != 1)) return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale) || !cap_ok(softcap)) return FA_ERR_INVALID_ARG;
  if (o_dtype != FA_BF16 && o_dtype != FA_FP32) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned256(workspace) ||
      !aligned16(k_new) || !aligned16(v_new) || !aligned4(seqlens) || !aligned4(starts) || !aligned4(lse) ||
      !aligned4(weights) || !aligned4(page_table) || !aligned4(slopes))
    return FA_ERR_INVALID_ARG;
  const float y = softcap > 0.f ? scale / softcap : 0.f;
  if (!std::isfinite(y) || !std::isfinite(softcap * fa::LOG2E)) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (paged && page_size % 16 != 0) return FA_ERR_UNSUPPORTED;
  const long long cap = static_cast<long long>(page_size) * pages_per_seq;
  if (cap + 1 > INT_MAX - 4096 || B > 65535 || Hkv > 65535) return FA_ERR_UNSUPPORTED;
  if (slopes != nullptr && cap + 1 >= (1 << 24)) return FA_ERR_UNSUPPORTED;
  if (weights != nullptr && weights_ld < cap) return FA_ERR_INVALID_ARG;
  const int rows = static_cast<int>(cap) + (append ? 1 : 0);
  if (workspace_bytes < fa_decode_scored_workspace_size(B, Hq, Hkv, rows, D, weights != nullptr))
    return FA_ERR_INVALID_ARG;
  const int G = Hq / Hkv;
  // heads of a fragment (rows past the group's heads are padding): one group of
  // up to eight heads reads its keys once
  const int GP = G == 1 ? 1 : G <= 4 ? 4 : 8;
  const long long HG = static_cast<long long>(Hkv) * ((G + GP - 1) / GP);
  const int chunk = scored_chunk(B, Hq, Hkv, rows);
  const int max_splits = (rows + chunk - 1) / chunk;
  if (!fits_int(B * HG * max_splits) || !fits_int(static_cast<long long>(B) * Hq)) return FA_ERR_UNSUPPORTED;
  const int sub_rows = (page_size % 32 == 0 || !paged) ? 32 : 16;
  CUtensorMap mk, mv;
  if (!map_bshd(&mk, k_cache, num_pages, page_size, Hkv, D, 64, sub_rows, true) ||
      !map_bshd(&mv, v_cache, num_pages, page_size, Hkv, D, 64, sub_rows, true))
    return FA_ERR_CUDA;
  char* ws = static_cast<char*>(workspace);
  const size_t lse_off = align_up(size_t(B) * Hq * max_splits * D * 4, 256);
  const size_t counter_off = lse_off + align_up(size_t(B) * Hq * max_splits * 4, 256);
  fa::DecParams p;
  p.seqlens = seqlens; p.q = static_cast<const uint16_t*>(q);
  p.k_new = static_cast<const uint16_t*>(k_new); p.v_new = static_cast<const uint16_t*>(v_new);
  p.k_cache = static_cast<uint16_t*>(k_cache);
  p.v_cache = static_cast<uint16_t*>(v_cache);
  p.page_table = page_table;
  p.o_part = reinterpret_cast<float*>(ws);
  p.lse_part = reinterpret_cast<float*>(ws + lse_off);
  p.work_counter = reinterpret_cast<int*>(ws + counter_off);
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.max_splits = max_splits; p.chunk = chunk;
  p.cap = static_cast<int>(cap); p.page_size = page_size; p.pages_per_seq = pages_per_seq; p.num_pages = num_pages;
  p.sub_rows = sub_rows;
  p.scale_log2 = scale * fa::LOG2E;
  p.wait_limit_ns = g_wait_limit_ns.load();
  p.y_scale = y; p.cap_log2 = softcap * fa::LOG2E; p.slopes = slopes; p.starts = starts;
  p.scores = weights != nullptr ? reinterpret_cast<float*>(ws + counter_off + 256) : nullptr;
  p.score_ld = static_cast<int>(align_up(size_t(rows), 4));
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(std::min<long long>(B * HG * max_splits, 3LL * sms));
  if (grid == B * HG * max_splits) p.work_counter = nullptr;   // one item per CTA at most
  else if (cudaMemsetAsync(p.work_counter, 0, sizeof(int), st_of(stream)) != cudaSuccess) return FA_ERR_CUDA;
  fa_status s;
  if (paged) s = append ? dispatch_decode_scored<true, true>(D, GP, mk, mv, p, grid, st_of(stream))
                        : dispatch_decode_scored<true, false>(D, GP, mk, mv, p, grid, st_of(stream));
  else s = append ? dispatch_decode_scored<false, true>(D, GP, mk, mv, p, grid, st_of(stream))
                  : dispatch_decode_scored<false, false>(D, GP, mk, mv, p, grid, st_of(stream));
  if (s != FA_OK) return s;
  fa::ScoredCombineParams c;
  c.o_part = p.o_part; c.lse_part = p.lse_part; c.scores = p.scores; c.weights = weights; c.o = o; c.lse = lse;
  c.d = p; c.o_fp32 = (o_dtype == FA_FP32); c.w_ld = weights_ld;
  const dim3 cgrid(G + (weights != nullptr ? (max_splits + fa::SCORED_RUN - 1) / fa::SCORED_RUN : 0), Hkv, B);
  auto* combine = D == 128 ? (append ? fa::scored_combine_kernel<128, true> : fa::scored_combine_kernel<128, false>)
                           : (append ? fa::scored_combine_kernel<64, true> : fa::scored_combine_kernel<64, false>);
  return launch_after(combine, cgrid, dim3(256), 0, st_of(stream), c);
}

size_t fa_key_weights_workspace_size(int B, int Hq, int Hkv, int Lq, int Lk) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || Lq < 0 || Lk < 0) return 0;
  const int parts = key_weight_parts(B, Hq, Hkv, Lq, Lk, kMaxSms);
  return fa_scored_workspace_size(B, Lq, Lk) +
         (parts > 1 ? size_t(parts) * B * Hkv * align_up(size_t(Lk), 128) * 4 : 0);
}

fa_status fa_key_weights(const void* q, const void* k, const float* lse, float* weights, int weights_ld,
                         int accumulate, int B, int Hq, int Hkv, int Lq, int Lk, int D, float scale, int causal,
                         const fa_score* score, void* workspace, size_t workspace_bytes, fa_stream_t stream) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Lq < 0 || Lk < 0 || Hq % Hkv != 0) return FA_ERR_INVALID_ARG;
  if (Lk > 0 && (!k || !weights || !workspace)) return FA_ERR_INVALID_ARG;
  if (Lk > 0 && Lq > 0 && (!q || !lse)) return FA_ERR_INVALID_ARG;
  if (!scale_ok(scale) || weights_ld < Lk) return FA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned4(lse) || !aligned4(weights) || !aligned256(workspace))
    return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  fa::KwParams p;
  int mod = fa::MOD_NONE;
  fa_status s = score_params(score, scale, causal, Lq, Lk, &p.sc, &mod);
  if (s != FA_OK) return s;
  const long long tiles = (static_cast<long long>(Lk) + 127) / 128 * B * Hkv;
  const long long pairs = (static_cast<long long>(Lq) + 127) / 128 * (Hq / Hkv);
  if (B > 65535 || !fits_int(tiles * 64) || !fits_int(pairs * 65)) return FA_ERR_UNSUPPORTED;
  if (Lk == 0) return FA_OK;
  if (workspace_bytes < fa_key_weights_workspace_size(B, Hq, Hkv, Lq, Lk)) return FA_ERR_INVALID_ARG;
  cudaStream_t st = st_of(stream);
  if (Lq == 0) {                                  // no query: every key gets nothing
    if (!accumulate && cudaMemset2DAsync(weights, size_t(weights_ld) * 4, 0, size_t(Lk) * 4, size_t(B) * Hkv, st) !=
                           cudaSuccess)
      return FA_ERR_CUDA;
    return FA_OK;
  }
  CUtensorMap mq, mk;
  if (!map_bshd(&mq, q, B, Lq, Hq, D, 64, 128, true) || !map_bshd(&mk, k, B, Lk, Hkv, D, 64, 128, true))
    return FA_ERR_CUDA;
  if ((s = launch_meta(&p.sc, B, Lq, Lk, workspace, st)) != FA_OK) return s;
  const int parts = key_weight_parts(B, Hq, Hkv, Lq, Lk, kMaxSms);
  float* part_sums = reinterpret_cast<float*>(static_cast<char*>(workspace) + fa_scored_workspace_size(B, Lq, Lk));
  p.lse = lse; p.out = parts > 1 ? part_sums : weights; p.ld = weights_ld; p.accumulate = accumulate != 0;
  p.B = B; p.Hq = Hq; p.Hkv = Hkv; p.Lq = Lq; p.Lk = Lk; p.parts = parts;
  p.num_items = static_cast<int>(tiles * parts);
  p.by_tile = fa::FastDiv::of(static_cast<uint32_t>(B * Hkv * parts));
  p.by_parts = fa::FastDiv::of(static_cast<uint32_t>(parts));
  p.by_hkv = fa::FastDiv::of(static_cast<uint32_t>(Hkv));
  p.by_group = fa::FastDiv::of(static_cast<uint32_t>(Hq / Hkv));
  p.scale_log2 = scale * fa::LOG2E;
  p.wait_limit_ns = g_wait_limit_ns.load();
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  const unsigned grid = static_cast<unsigned>(std::min(p.num_items, sms));
  s = with_mod(mod, [&](auto m) {
    return D == 128 ? launch_kw<128, decltype(m)::value>(mq, mk, p, grid, st)
                    : launch_kw<64, decltype(m)::value>(mq, mk, p, grid, st);
  });
  if (s != FA_OK || parts == 1) return s;
  const size_t n = size_t(B) * Hkv * Lk;
  return launch_after(fa::kw_reduce_kernel, dim3(static_cast<unsigned>(std::min<size_t>((n + 255) / 256, size_t(sms) * 16))),
                      dim3(256), 0, st, static_cast<const float*>(part_sums), weights, parts, B * Hkv, Lk, weights_ld,
                      static_cast<int>(accumulate != 0));
}

fa_status fa_cache_evict(const fa_kv_rows* src, const fa_kv_rows* dst, const float* weights_src, int weights_src_ld,
                         float* weights_dst, int weights_dst_ld, const int* seqlens_src, int* seqlens_dst, int* kept,
                         int B, int Hkv, int D, int keep, int recent, fa_stream_t stream) {
  if (!src || !dst || !weights_src || !weights_dst || !seqlens_src || !seqlens_dst || !kept) return FA_ERR_INVALID_ARG;
  if (B <= 0 || Hkv <= 0 || D <= 0 || keep <= 0 || recent < 0 || recent > keep) return FA_ERR_INVALID_ARG;
  if (!aligned4(weights_src) || !aligned4(weights_dst) || !aligned4(seqlens_src) || !aligned4(seqlens_dst) ||
      !aligned4(kept))
    return FA_ERR_INVALID_ARG;
  long long rows[2];
  const fa_kv_rows* side[2] = {src, dst};
  for (int i = 0; i < 2; ++i) {
    const fa_kv_rows* r = side[i];
    if (!r->k || !r->v || !aligned16(r->k) || !aligned16(r->v) || r->k == r->v || r->page_size <= 0)
      return FA_ERR_INVALID_ARG;
    if (!aligned4(r->page_table) || (r->page_table && (r->pages_per_seq <= 0 || r->num_pages <= 0)))
      return FA_ERR_INVALID_ARG;
    rows[i] = r->page_table ? static_cast<long long>(r->page_size) * r->pages_per_seq : r->page_size;
  }
  if (keep > rows[1] || weights_src_ld < rows[0] || weights_dst_ld < keep) return FA_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > 4096 || B > 65535 || Hkv > 32767) return FA_ERR_UNSUPPORTED;
  if (rows[0] > INT_MAX - 65536 || rows[1] > INT_MAX - 65536 || !fits_int(static_cast<long long>(B) * Hkv))
    return FA_ERR_UNSUPPORTED;
  const bool in_place = src->k == dst->k || src->v == dst->v;
  if (in_place && (src->k != dst->k || src->v != dst->v || src->page_table != dst->page_table ||
                   src->page_size != dst->page_size ||
                   (src->page_table && (src->pages_per_seq != dst->pages_per_seq || src->num_pages != dst->num_pages))))
    return FA_ERR_INVALID_ARG;
  // extents in bytes: what does not name the same tensor must not overlap it
  auto bytes = [&](const fa_kv_rows* r) {
    const size_t n = r->page_table ? size_t(r->num_pages) * r->page_size : size_t(B) * r->page_size;
    return n * Hkv * D * 2;
  };
  if (!in_place)
    for (const void* a : {src->k, src->v})
      for (const void* b : {dst->k, dst->v})
        if (overlap(a, bytes(src), b, bytes(dst))) return FA_ERR_INVALID_ARG;
  if (weights_src == weights_dst ? weights_src_ld != weights_dst_ld
                                 : overlap(weights_src, size_t(B) * Hkv * weights_src_ld * 4, weights_dst,
                                           size_t(B) * Hkv * weights_dst_ld * 4))
    return FA_ERR_INVALID_ARG;
  if (seqlens_src != seqlens_dst && overlap(seqlens_src, size_t(B) * 4, seqlens_dst, size_t(B) * 4))
    return FA_ERR_INVALID_ARG;
  cudaStream_t st = st_of(stream);
  fa::EvictParams p;
  auto fill = [](const fa_kv_rows* r, long long n) {
    fa::KvRows o;
    o.k = static_cast<uint16_t*>(r->k); o.v = static_cast<uint16_t*>(r->v); o.table = r->page_table;
    o.cap = static_cast<int>(n); o.page_size = r->page_size; o.pages_per_seq = r->pages_per_seq;
    o.num_pages = r->num_pages;
    return o;
  };
  p.src = fill(src, rows[0]);
  p.dst = fill(dst, rows[1]);
  p.w_src = weights_src; p.w_dst = weights_dst; p.len_src = seqlens_src; p.len_dst = seqlens_dst; p.kept = kept;
  p.B = B; p.Hkv = Hkv; p.D = D; p.keep = keep; p.recent = recent;
  p.w_src_ld = weights_src_ld; p.w_dst_ld = weights_dst_ld;
  const int sms = sm_count();
  if (sms <= 0) return FA_ERR_CUDA;
  // a slice is a power of two of 16-byte chunks: the whole row where blocks own
  // rows; in place, narrower (down to a 32-byte sector) until the SMs are filled
  int chunks = 1;
  while (chunks < D / 8 && chunks < fa::EVICT_MOVE_THREADS) chunks *= 2;
  while (in_place && chunks > 2 && 2LL * B * Hkv * ((D / 8 + chunks - 1) / chunks) < 4LL * sms) chunks /= 2;
  p.slice_chunks = chunks;
  p.cached = std::min(p.src.cap, fa::EVICT_CACHED);
  const size_t key_bytes = align_up(size_t(p.cached) * 4, 16);
  static std::atomic<uint64_t> attr_done{0};
  if (!ensure_smem_attr(fa::evict_select_kernel, fa::EVICT_CACHED * 4, attr_done)) return FA_ERR_CUDA;
  fa::evict_select_kernel<<<B * Hkv, fa::EVICT_THREADS, key_bytes, st>>>(p);
  if (launch_status() != FA_OK) return FA_ERR_CUDA;
  const int slices = (D / 8 + chunks - 1) / chunks, step = fa::EVICT_MOVE_THREADS / chunks * fa::EVICT_UNROLL;
  const dim3 grid(in_place ? slices : slices * ((keep + step - 1) / step), 2 * Hkv, B);
  return launch_after(in_place ? fa::evict_move_kernel<true> : fa::evict_move_kernel<false>, grid,
                      dim3(fa::EVICT_MOVE_THREADS), 0, st, p);
}

fa_status fa_device_status(int* code, int* where, int reset, fa_stream_t stream) {
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  uint32_t s = 0, w = 0;
  if (cudaMemcpyFromSymbolAsync(&s, fa::g_fa_dev_status, 4, 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaMemcpyFromSymbolAsync(&w, fa::g_fa_dev_where, 4, 0, cudaMemcpyDeviceToHost, st) != cudaSuccess ||
      cudaStreamSynchronize(st) != cudaSuccess)
    return FA_ERR_CUDA;
  if (code)
    *code = (s == fa::FA_DEV_TIMEOUT)     ? FA_ERR_TIMEOUT
            : (s == fa::FA_DEV_BAD_INPUT) ? FA_ERR_INVALID_ARG
            : (s == fa::FA_DEV_BAD_INDEX) ? FA_ERR_DEVICE_INDEX
                                          : FA_OK;
  if (where) *where = static_cast<int>(w);
  if (reset) {
    const uint32_t zero = 0;
    if (cudaMemcpyToSymbolAsync(fa::g_fa_dev_status, &zero, 4, 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaMemcpyToSymbolAsync(fa::g_fa_dev_where, &zero, 4, 0, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaStreamSynchronize(st) != cudaSuccess)
      return FA_ERR_CUDA;
  }
  return FA_OK;
}

fa_status fa_launch_guard(int bwd, int D, int causal, int* num_regs, int* expected_regs, int* state) {
  // D = -128 names the e4m3 forward
  const bool fp8 = (D == -128 && !bwd);
  if (D != 64 && D != 128 && !fp8) return FA_ERR_INVALID_ARG;
  const int slot = kernel_slot(bwd != 0, D, causal != 0, fp8);
  if (state) *state = g_regs_state[slot].load();
  if (expected_regs) *expected_regs = bwd ? fa::BWD_LAUNCH_REGS : fa::FWD_LAUNCH_REGS;
  if (num_regs) {
    cudaFuncAttributes a;
    cudaError_t e;
    if (fp8) {
      e = causal ? cudaFuncGetAttributes(&a, fa::fwd_kernel<128, true, true>)
                 : cudaFuncGetAttributes(&a, fa::fwd_kernel<128, false, true>);
    } else if (bwd) {
      e = D == 128 ? (causal ? cudaFuncGetAttributes(&a, fa::bwd_main_kernel<128, true>)
                             : cudaFuncGetAttributes(&a, fa::bwd_main_kernel<128, false>))
                   : (causal ? cudaFuncGetAttributes(&a, fa::bwd_main_kernel<64, true>)
                             : cudaFuncGetAttributes(&a, fa::bwd_main_kernel<64, false>));
    } else {
      e = D == 128 ? (causal ? cudaFuncGetAttributes(&a, fa::fwd_kernel<128, true>)
                             : cudaFuncGetAttributes(&a, fa::fwd_kernel<128, false>))
                   : (causal ? cudaFuncGetAttributes(&a, fa::fwd_kernel<64, true>)
                             : cudaFuncGetAttributes(&a, fa::fwd_kernel<64, false>));
    }
    if (e != cudaSuccess) return FA_ERR_CUDA;
    *num_regs = a.numRegs;
  }
  return FA_OK;
}

fa_status fa_selftest_exp2_poly(const float* x, float* y, int n, fa_stream_t stream) {
  if (!x || !y || n < 0) return FA_ERR_INVALID_ARG;
  if (n == 0) return FA_OK;
  const int threads = 256, pairs = (n + 1) / 2;
  selftest_exp2_poly_kernel<<<(pairs + threads - 1) / threads, threads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(x, y, n);
  return launch_status();
}

fa_status fa_selftest_wait_timeout(unsigned long long wait_ns, fa_stream_t stream) {
  if (wait_ns == 0 || wait_ns > 10000000000ull) return FA_ERR_INVALID_ARG;
  selftest_wait_kernel<<<1, 32, 0, reinterpret_cast<cudaStream_t>(stream)>>>(wait_ns);
  return launch_status();
}

}  // extern "C"
