// Mixture-of-experts glue around the products grouped by expert: the router
// (softmax, top-k, grouping of the tokens by expert), the weighted
// combination of the experts' outputs, and the whole sparse MLP block.
//
// The Unweight page compresses the matrices of dense MLPs; a sparse MLP holds
// the same three matrices once per expert.  The block is not on the page.
#include <algorithm>
#include <cfloat>
#include <cstring>

#include "uw_device.cuh"
#include "uw_internal.h"

namespace uw {

namespace {

// ------------------------------- router --------------------------------------
// LPT lanes per token, the token's logits in registers (EPL per lane: expert
// lane + LPT i).  Each of the top_k steps finds the largest remaining logit
// with one reduction over the lanes and the lowest expert that has it with a
// second; the tokens of a block that chose an expert are a bit mask in shared memory,
// so a token's place among them is a population count, whatever the order of
// the atomics.
//
// A prompt takes two launches: the first chooses, counts per block and finds
// each choice's place among its block's, the second adds up the counts of the
// blocks before it (at most kMaxRouteBlocks).  Up to 64 tokens take one block
// and one launch (128 tokens in one block: 64 experts, top 8, 10.1 us against
// 8.5).  Launch latency bounds both: 8192 x 64 BF16 logits are 1 MB.
constexpr int kRouteWarps = 16, kRouteThreads = 32 * kRouteWarps;
constexpr int kRouteChunk = 64;       // tokens ranked together (two mask words)
constexpr int kMaxRouteBlocks = 128;  // a block ranks as many chunks as that needs

struct RouteParams {
  const void* logits;
  int fp32, T, E, k, renormalize;
  int tokens_per_block;
  float* weights;
  int32_t* experts;
  int32_t* slots;
  int32_t* rows;
  int32_t* offsets;
  int32_t* counts;  // [blocks][E]
};

// Ordered key of a logit: larger logit, larger key; 0 for one that can never
// be chosen (-inf, NaN).  +inf counts as the largest finite value.
__device__ __forceinline__ uint32_t logit_key(float v) {
  if (!(v > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(fminf(v, FLT_MAX) + 0.0f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? key ^ 0x80000000u : ~key);
}

// Largest / smallest over the LPT lanes of a token.
template <int LPT>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  if constexpr (LPT == 32) {
    return __reduce_max_sync(0xFFFFFFFFu, v);
  } else {
#pragma unroll
    for (int d = LPT / 2; d; d >>= 1) v = max(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
  }
}
template <int LPT>
__device__ __forceinline__ uint32_t lanes_min(uint32_t v) {
  if constexpr (LPT == 32) {
    return __reduce_min_sync(0xFFFFFFFFu, v);
  } else {
#pragma unroll
    for (int d = LPT / 2; d; d >>= 1) v = min(v, __shfl_xor_sync(0xFFFFFFFFu, v, d));
    return v;
  }
}

// Chooses token t's experts (every lane of the warp takes part; t < 0: a lane
// group without a token).  masks: the block's bit masks, `bit` this token's.
template <int EPL, int LPT>
__device__ __forceinline__ void choose(const RouteParams& p, int t, uint32_t* masks, uint32_t word, uint32_t bit) {
  constexpr int kMine = (UW_MAX_TOP_K + LPT - 1) / LPT;
  const int sub = threadIdx.x & (LPT - 1);
  uint32_t key[EPL];
  const int64_t base = static_cast<int64_t>(t) * p.E;
  // all loads leave before the first is used (past the last expert the last
  // one again); a lane group without a token reads token 0
  float v[EPL];
  if (p.fp32) {
    const float* src = static_cast<const float*>(p.logits) + max(base, int64_t(0));
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = src[min(sub + LPT * i, p.E - 1)];
  } else {
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.logits) + max(base, int64_t(0));
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = __bfloat162float(src[min(sub + LPT * i, p.E - 1)]);
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) key[i] = t >= 0 && sub + LPT * i < p.E ? logit_key(v[i]) : 0u;
  uint32_t local = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) local = max(local, key[i]);
  const uint32_t top = lanes_max<LPT>(local);
  const float vmax = key_logit(top);
  float whole = 0.0f;  // sum of exp(l - max), over all experts or over the chosen
  if (!p.renormalize) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) whole += key[i] ? expf(key_logit(key[i]) - vmax) : 0.0f;
#pragma unroll
    for (int d = LPT / 2; d; d >>= 1) whole += __shfl_xor_sync(0xFFFFFFFFu, whole, d);
  }
  // lane s of the token keeps choices s, s + LPT, ..
  float mine[kMine];
  int chosen[kMine];
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    mine[q] = 0.0f;
    chosen[q] = -1;
  }
  uint32_t best = top;
  for (int j = 0; j < p.k; ++j) {
    if (j) {
      local = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) local = max(local, key[i]);
      best = lanes_max<LPT>(local);
    }
    uint32_t at = 0xFFFFFFFFu;  // the lowest expert that has it
#pragma unroll
    for (int i = EPL - 1; i >= 0; --i)
      if (key[i] == best) at = static_cast<uint32_t>(sub + LPT * i);
    at = lanes_min<LPT>(at);
    const bool any = best != 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (any && at == static_cast<uint32_t>(sub + LPT * i)) key[i] = 0;
    const float e = any ? expf(key_logit(best) - vmax) : 0.0f;
    if (p.renormalize) whole += e;
#pragma unroll
    for (int q = 0; q < kMine; ++q)
      if (any && j == q * LPT + sub) {
        mine[q] = e;
        chosen[q] = static_cast<int>(at);
      }
  }
  if (t < 0) return;
#pragma unroll
  for (int q = 0; q < kMine; ++q) {
    const int j = q * LPT + sub;
    if (j < p.k) {
      const int64_t i = static_cast<int64_t>(t) * p.k + j;
      p.experts[i] = chosen[q];
      p.weights[i] = chosen[q] < 0 ? 0.0f : mine[q] / whole;
      if (chosen[q] >= 0) atomicOr(&masks[2 * chosen[q] + word], bit);
    }
  }
}

// Exclusive scan of total[0..E) into first[0..E]; one warp.
__device__ __forceinline__ void scan_experts(const int32_t* total, int32_t* first, int E, int lane) {
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int v = e0 + lane < E ? total[e0 + lane] : 0;
    int incl = v;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int u = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += u;
    }
    if (e0 + lane < E) first[e0 + lane] = base + incl - v;
    base += __shfl_sync(0xFFFFFFFFu, incl, 31);
  }
  if (lane == 0) first[E] = base;
}

// The places of the tokens [t0, t0 + n) among the choices of their experts,
// from their masks and the choices counted before them.
__device__ __forceinline__ void place(const RouteParams& p, int t0, int n, const uint32_t* masks, const int32_t* base) {
  for (int i = threadIdx.x; i < n * p.k; i += kRouteThreads) {
    const int t = i / p.k;
    const int64_t at = static_cast<int64_t>(t0) * p.k + i;
    const int e = p.experts[at];
    int slot = -1;
    if (e >= 0) {
      const uint32_t lo = masks[2 * e], hi = masks[2 * e + 1];
      slot = base[e] + (t < 32 ? __popc(lo & ((1u << t) - 1)) : __popc(lo) + __popc(hi & ((1u << (t - 32)) - 1)));
    }
    p.slots[at] = slot;
  }
}

// Turns the places of the tokens [t0, t0 + n) into slots: each expert's choices
// of this block start at base[e].
__device__ __forceinline__ void settle(const RouteParams& p, int t0, int n, const int32_t* base) {
  const int64_t i0 = static_cast<int64_t>(t0) * p.k;
  for (int i = threadIdx.x; i < n * p.k; i += kRouteThreads) {
    const int e = p.experts[i0 + i];
    if (e < 0) continue;
    const int slot = base[e] + p.slots[i0 + i];
    p.slots[i0 + i] = slot;
    p.rows[slot] = t0 + i / p.k;
  }
}

// Chooses the experts of a block's tokens.  ONE: the only block, which places
// them too; else the block's counts go to the workspace.
template <int EPL, int LPT, bool ONE>
__global__ void __launch_bounds__(kRouteThreads) route_kernel(const RouteParams p) {
  extern __shared__ int32_t sh[];
  uint32_t* masks = reinterpret_cast<uint32_t*>(sh);  // [E][2]
  int32_t* total = sh + 2 * p.E;                      // [E]
  int32_t* first = total + p.E;                       // [E + 1]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
    masks[2 * e] = masks[2 * e + 1] = 0;
    total[e] = 0;
  }
  griddep_wait();
  griddep_launch_dependents();
  const int t0 = blockIdx.x * p.tokens_per_block, t1 = min(p.T, t0 + p.tokens_per_block);
  __syncthreads();
  for (int c = t0; c < t1; c += kRouteChunk) {
    constexpr int kTokens = kRouteThreads / LPT;  // chosen for at a time
    for (int i0 = 0; i0 < min(kRouteChunk, t1 - c); i0 += kTokens) {
      const int i = i0 + static_cast<int>(threadIdx.x) / LPT;
      if (i0 + warp * (32 / LPT) >= min(kRouteChunk, t1 - c)) break;  // no token in the whole warp
      choose<EPL, LPT>(p, c + i < t1 ? c + i : -1, masks, static_cast<uint32_t>(i >> 5), 1u << (i & 31));
    }
    __syncthreads();
    place(p, c, min(kRouteChunk, t1 - c), masks, total);
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) {
      total[e] += __popc(masks[2 * e]) + __popc(masks[2 * e + 1]);
      masks[2 * e] = masks[2 * e + 1] = 0;
    }
    __syncthreads();
  }
  if constexpr (ONE) {
    if (warp == 0) scan_experts(total, first, p.E, lane);
    __syncthreads();
    for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) p.offsets[e] = first[e];
    settle(p, 0, p.T, first);
  } else {
    for (int e = threadIdx.x; e < p.E; e += kRouteThreads) p.counts[static_cast<int64_t>(blockIdx.x) * p.E + e] = total[e];
  }
}

// Adds up the counts of the blocks before this one and turns the places among
// a block's choices into slots.
__global__ void __launch_bounds__(kRouteThreads) place_kernel(const RouteParams p) {
  extern __shared__ int32_t sh[];
  int32_t* total = sh;              // [E]
  int32_t* first = total + p.E;     // [E + 1]
  int32_t* base = first + p.E + 1;  // [E] choices of earlier blocks, then the block's first slots
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += kRouteThreads) total[e] = base[e] = 0;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  // several threads per expert, each a run of blocks; integer sums, so the
  // order of the shared-memory atomics does not matter
  const int parts = max(1, kRouteThreads / p.E);
  for (int i = threadIdx.x; i < parts * p.E; i += kRouteThreads) {
    const int e = i % p.E, part = i / p.E;
    int all = 0, earlier = 0;
#pragma unroll 16
    for (int b = part; b < static_cast<int>(gridDim.x); b += parts) {
      const int v = __ldcg(p.counts + static_cast<int64_t>(b) * p.E + e);
      all += v;
      if (b < static_cast<int>(blockIdx.x)) earlier += v;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&base[e], earlier);
  }
  __syncthreads();
  if (warp == 0) scan_experts(total, first, p.E, lane);
  __syncthreads();
  for (int e = threadIdx.x; e <= p.E; e += kRouteThreads) {
    if (blockIdx.x == 0) p.offsets[e] = first[e];
    if (e < p.E) base[e] += first[e];
  }
  __syncthreads();
  const int t0 = static_cast<int>(blockIdx.x) * p.tokens_per_block;
  settle(p, t0, min(p.T - t0, p.tokens_per_block), base);
}

// Launch with programmatic dependent launch: every kernel here waits for the
// one ahead before it touches memory that one may use.
template <typename... Args>
uw_status launch_pdl(void (*kernel)(Args...), unsigned grid, unsigned block, size_t smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t err = cudaLaunchKernelEx(&cfg, kernel, args...);
  note_launch();
  if (err != cudaSuccess) return cuda_status(err);
  return cuda_status(cudaGetLastError());
}

struct RoutePlan {
  int blocks = 1, tokens_per_block = kRouteChunk;
  size_t bytes = 0;
};
bool route_plan(int64_t T, int64_t E, int64_t k, RoutePlan* out) {
  if (T < 0 || T > UW_MAX_TOKENS || E < 1 || E > kMaxExperts || k < 1 || k > E || k > UW_MAX_TOP_K) return false;
  RoutePlan r;
  const int64_t chunks = std::max<int64_t>(1, (T + kRouteChunk - 1) / kRouteChunk);
  const int64_t per = (chunks + kMaxRouteBlocks - 1) / kMaxRouteBlocks;
  r.tokens_per_block = static_cast<int>(per * kRouteChunk);
  r.blocks = static_cast<int>((chunks + per - 1) / per);
  // (the blocks that the counts have room for never fall with T)
  const int64_t most = std::min<int64_t>(chunks, kMaxRouteBlocks);
  r.bytes = kWsHeader + kCounterBytes + (most > 1 ? align_up(static_cast<size_t>(most) * E * 4, 256) : 0);
  *out = r;
  return true;
}

template <int EPL, int LPT>
uw_status launch_route_epl(const RouteParams& p, const RoutePlan& r, cudaStream_t s) {
  const size_t smem = static_cast<size_t>(4 * p.E + 1) * 4;
  if (r.blocks == 1) return launch_pdl(route_kernel<EPL, LPT, true>, 1u, kRouteThreads, smem, s, p);
  return launch_pdl(route_kernel<EPL, LPT, false>, static_cast<unsigned>(r.blocks), kRouteThreads, smem, s, p);
}

uw_status launch_route(const RouteParams& p, const RoutePlan& r, cudaStream_t s) {
  // up to 256 experts: 8 lanes per token, so that a warp chooses for 4 tokens
  // at once (against a warp per token: 8192 x 64 logits 13.1 / 15.2 us, 1000 x
  // 256 13.9 / 16.2, 20000 x 256 41 / 45, 8192 x 256 24 / 21); more: a warp
  uw_status st;
  if (p.E <= 8) st = launch_route_epl<1, 8>(p, r, s);
  else if (p.E <= 16) st = launch_route_epl<2, 8>(p, r, s);
  else if (p.E <= 32) st = launch_route_epl<4, 8>(p, r, s);
  else if (p.E <= 64) st = launch_route_epl<8, 8>(p, r, s);
  else if (p.E <= 128) st = launch_route_epl<16, 8>(p, r, s);
  else if (p.E <= 256) st = launch_route_epl<32, 8>(p, r, s);
  else st = launch_route_epl<kMaxExperts / 32, 32>(p, r, s);
  if (st != UW_OK || r.blocks == 1) return st;
  return launch_pdl(place_kernel, static_cast<unsigned>(r.blocks), kRouteThreads, static_cast<size_t>(3 * p.E + 1) * 4,
                    s, p);
}

// ------------------------------- combine -------------------------------------
// y[t] = r[t] + sum_j w[t, j] part[slots[t, j]], FP32 sums in order of j, one
// rounding.  Bound by HBM: every part is read once.  A thread owns VEC
// consecutive columns of one token (8 where rows start on 16 bytes), or four
// single ones 256 apart, and has the loads of up to four parts in flight
// (3132 tokens, 955 columns: 7.6 us, 15.2 with one column per thread).
struct CombineParams {
  const void* parts;
  const int32_t* slots;
  const float* weights;
  const __nv_bfloat16* residual;
  __nv_bfloat16* y;
  int T, k, cols, n_rows, col_blocks;
};

// VEC consecutive values (8) from 16-byte loads.
template <int VEC, bool FP32>
__device__ __forceinline__ void load_part(const void* parts, int64_t i, float (&v)[VEC]) {
  if constexpr (FP32) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(parts) + i);
#pragma unroll
    for (int q = 0; q < VEC / 4; ++q) {
      const float4 f = __ldcs(src + q);
      v[4 * q] = f.x;
      v[4 * q + 1] = f.y;
      v[4 * q + 2] = f.z;
      v[4 * q + 3] = f.w;
    }
  } else {
    const uint4 u = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(parts) + i));
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[2 * q] = __uint_as_float(w[q] << 16);
      v[2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  }
}

template <int VEC, bool FP32>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p) {
  constexpr int kCols = VEC == 1 ? 4 : VEC;  // columns per thread
  griddep_wait();
  griddep_launch_dependents();
  const int t = blockIdx.x / p.col_blocks;
  const int c = (blockIdx.x - t * p.col_blocks) * 256 * kCols + threadIdx.x * VEC;
  if (c >= p.cols) return;
  const int64_t at = static_cast<int64_t>(t) * p.cols + c;
  const int32_t* slots = p.slots + static_cast<int64_t>(t) * p.k;
  const float* weights = p.weights + static_cast<int64_t>(t) * p.k;
  // the thread's columns of the row that starts with element i - c
  auto load = [&](const void* rows, bool fp32, int64_t i, float (&v)[kCols]) {
    if constexpr (VEC == 1) {
#pragma unroll
      for (int q = 0; q < kCols; ++q) {
        const int64_t k = i + 256 * q;
        if (c + 256 * q >= p.cols) v[q] = 0.0f;
        else v[q] = fp32 ? __ldcs(static_cast<const float*>(rows) + k)
                         : __bfloat162float(static_cast<const __nv_bfloat16*>(rows)[k]);
      }
    } else if (fp32) {
      load_part<VEC, true>(rows, i, v);
    } else {
      load_part<VEC, false>(rows, i, v);
    }
  };
  float acc[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.0f;
  for (int j0 = 0; j0 < p.k; j0 += 4) {
    float v[4][kCols], w[4];
    bool have[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int s = j0 + q < p.k ? slots[j0 + q] : -1;
      have[q] = s >= 0 && s < p.n_rows;
      if (have[q]) {
        w[q] = weights[j0 + q];
        load(p.parts, FP32, static_cast<int64_t>(s) * p.cols + c, v[q]);
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q)
      if (have[q])
#pragma unroll
        for (int i = 0; i < kCols; ++i) acc[i] = fmaf(w[q], v[q][i], acc[i]);
  }
  if (p.residual) {
    float r[kCols];
    load(p.residual, false, at, r);
#pragma unroll
    for (int i = 0; i < kCols; ++i) acc[i] += r[i];
  }
  if constexpr (VEC == 1) {
#pragma unroll
    for (int q = 0; q < kCols; ++q)
      if (c + 256 * q < p.cols) p.y[at + 256 * q] = __float2bfloat16_rn(acc[q]);
  } else {
    uint32_t o[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * q], acc[2 * q + 1]);
      o[q] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p.y + at) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

uw_status launch_combine(const void* parts, int fp32, const int32_t* slots, const float* weights, int32_t T, int32_t k,
                         int64_t cols, int32_t n_rows, const uint16_t* residual, uint16_t* y, cudaStream_t s) {
  if (T < 0 || T > UW_MAX_TOKENS || k < 1 || k > UW_MAX_TOP_K || n_rows < 0 || cols < 1) return UW_ERR_INVALID_ARG;
  if (fp32 != UW_OUT_BF16 && fp32 != UW_OUT_FP32) return UW_ERR_INVALID_ARG;
  if (T == 0) return UW_OK;
  if ((!parts && n_rows > 0) || !slots || !weights || !y || !aligned_to(parts, fp32 ? 4 : 2) || !aligned_to(slots, 4) ||
      !aligned_to(weights, 4) || !aligned_to(residual, 2) || !aligned_to(y, 2))
    return UW_ERR_INVALID_ARG;
  // 16-byte accesses where every row starts on 16 bytes, else one value each
  const int vec = cols % 8 == 0 && aligned16(parts) && aligned16(residual) && aligned16(y) ? 8 : 1;
  const int64_t per_block = 256 * (vec == 8 ? 8 : 4);
  const int64_t col_blocks = (cols + per_block - 1) / per_block;
  if (cols > (int64_t(1) << 30) || col_blocks * T > 0x7FFFFFFF) return UW_ERR_UNSUPPORTED_SHAPE;
  DeviceInfo dev;
  const uw_status st = device_info(&dev);
  if (st != UW_OK) return st;
  CombineParams p;
  p.parts = parts;
  p.slots = slots;
  p.weights = weights;
  p.residual = reinterpret_cast<const __nv_bfloat16*>(residual);
  p.y = reinterpret_cast<__nv_bfloat16*>(y);
  p.T = T;
  p.k = k;
  p.cols = static_cast<int>(cols);
  p.n_rows = n_rows;
  p.col_blocks = static_cast<int>(col_blocks);
  const unsigned grid = static_cast<unsigned>(col_blocks * T);
  if (vec == 8)
    return fp32 ? launch_pdl(combine_kernel<8, true>, grid, 256, 0, s, p)
                : launch_pdl(combine_kernel<8, false>, grid, 256, 0, s, p);
  return fp32 ? launch_pdl(combine_kernel<1, true>, grid, 256, 0, s, p)
              : launch_pdl(combine_kernel<1, false>, grid, 256, 0, s, p);
}

uw_status route(const void* logits, int32_t logits_type, int32_t T, int32_t E, int32_t k, int32_t renormalize,
                float* weights, int32_t* experts, int32_t* slots, int32_t* rows, int32_t* offsets, void* ws,
                size_t ws_bytes, cudaStream_t s) {
  RoutePlan r;
  if (!route_plan(T, E, k, &r) || (logits_type != UW_OUT_BF16 && logits_type != UW_OUT_FP32)) return UW_ERR_INVALID_ARG;
  if (!offsets || !ws || !aligned_to(offsets, 4) || !aligned16(ws)) return UW_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !weights || !experts || !slots || !rows ||
                !aligned_to(logits, logits_type == UW_OUT_FP32 ? 4 : 2) || !aligned_to(weights, 4) ||
                !aligned_to(experts, 4) || !aligned_to(slots, 4) || !aligned_to(rows, 4)))
    return UW_ERR_INVALID_ARG;
  if (ws_bytes < r.bytes) return UW_ERR_WORKSPACE_TOO_SMALL;
  DeviceInfo dev;
  const uw_status st = device_info(&dev);
  if (st != UW_OK) return st;
  RouteParams p;
  p.logits = logits;
  p.fp32 = logits_type == UW_OUT_FP32;
  p.T = T;
  p.E = E;
  p.k = k;
  p.renormalize = renormalize != 0;
  p.tokens_per_block = r.tokens_per_block;
  p.weights = weights;
  p.experts = experts;
  p.slots = slots;
  p.rows = rows;
  p.offsets = offsets;
  p.counts = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kWsHeader + kCounterBytes);
  return launch_route(p, r, s);
}

// Workspace of the block: the largest grouped product's (the router's counts
// share it), then the routing, the hidden rows and the experts' outputs.
struct MoeWs {
  size_t base = 0, weights = 0, experts = 0, slots = 0, rows = 0, offsets = 0, h = 0, parts = 0, total = 0;
};
bool moe_ws(const uw_experts* gate, const uw_experts* up, const uw_experts* down, int64_t T, int64_t k, MoeWs* out) {
  if (!gate || !up || !down) return false;
  if (up->n_experts != gate->n_experts || down->n_experts != gate->n_experts || up->rows != gate->rows ||
      up->cols != gate->cols || down->rows != gate->cols || down->cols != gate->rows)
    return false;
  RoutePlan r;
  if (!route_plan(T, gate->n_experts, k, &r)) return false;
  const int64_t n = T * k;
  if (n > UW_MAX_SLOTS) return false;
  const size_t a = grouped_ws_bytes(gate->rows, gate->cols, gate->n_experts, static_cast<int>(n), true, true);
  const size_t b = grouped_ws_bytes(down->rows, down->cols, gate->n_experts, static_cast<int>(n), false, false);
  if (!a || !b) return false;
  MoeWs w;
  size_t at = align_up(std::max({a, b, r.bytes}), 256);
  w.base = at;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align_up(std::max<size_t>(bytes, 1), 256);
    return here;
  };
  w.weights = take(static_cast<size_t>(n) * 4);
  w.experts = take(static_cast<size_t>(n) * 4);
  w.slots = take(static_cast<size_t>(n) * 4);
  w.rows = take(static_cast<size_t>(n) * 4);
  w.offsets = take(static_cast<size_t>(gate->n_experts + 1) * 4);
  w.h = take(static_cast<size_t>(n) * gate->rows * 2);
  w.parts = take(static_cast<size_t>(n) * down->rows * 4);
  w.total = at;
  *out = w;
  return true;
}

}  // namespace
}  // namespace uw

using namespace uw;

extern "C" size_t uw_moe_route_workspace_bytes(int32_t n_tokens, int32_t n_experts, int32_t top_k) {
  RoutePlan r;
  return route_plan(n_tokens, n_experts, top_k, &r) ? r.bytes : 0;
}

extern "C" uw_status uw_moe_route(const void* logits, int32_t logits_type, int32_t n_tokens, int32_t n_experts,
                                  int32_t top_k, int32_t renormalize, float* weights, int32_t* experts, int32_t* slots,
                                  int32_t* rows, int32_t* offsets, void* ws, size_t ws_bytes, void* stream) {
  return route(logits, logits_type, n_tokens, n_experts, top_k, renormalize, weights, experts, slots, rows, offsets, ws,
               ws_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" uw_status uw_moe_combine(const void* parts, int32_t parts_type, const int32_t* slots, const float* weights,
                                    int32_t n_tokens, int32_t top_k, int64_t cols, int32_t n_rows,
                                    const uint16_t* residual, uint16_t* y, void* stream) {
  return launch_combine(parts, parts_type, slots, weights, n_tokens, top_k, cols, n_rows, residual, y,
                        static_cast<cudaStream_t>(stream));
}

extern "C" size_t uw_moe_workspace_bytes(const uw_experts* gate, const uw_experts* up, const uw_experts* down,
                                         int32_t n_tokens, int32_t top_k) {
  MoeWs w;
  return moe_ws(gate, up, down, n_tokens, top_k, &w) ? w.total : 0;
}

extern "C" uw_status uw_moe_block(const uw_experts* gate, const uw_experts* up, const uw_experts* down,
                                  const void* logits, int32_t logits_type, int32_t top_k, int32_t renormalize,
                                  const uint16_t* x, int32_t n_tokens, const uint16_t* residual, uint16_t* y, void* ws,
                                  size_t ws_bytes, void* stream) {
  MoeWs w;
  if (!moe_ws(gate, up, down, n_tokens, top_k, &w)) return UW_ERR_INVALID_ARG;
  if (!gate->table || !up->table || !down->table || !ws || !aligned16(ws)) return UW_ERR_INVALID_ARG;
  if (n_tokens == 0) return UW_OK;
  if (!x || !y || !logits || !aligned16(x) || !aligned_to(y, 2) || !aligned_to(residual, 2)) return UW_ERR_INVALID_ARG;
  if (ws_bytes < w.total) return UW_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  float* weights = reinterpret_cast<float*>(base + w.weights);
  int32_t* slots = reinterpret_cast<int32_t*>(base + w.slots);
  int32_t* rows = reinterpret_cast<int32_t*>(base + w.rows);
  int32_t* offsets = reinterpret_cast<int32_t*>(base + w.offsets);
  const int32_t n = n_tokens * top_k;
  uw_status st = route(logits, logits_type, n_tokens, gate->n_experts, top_k, renormalize, weights,
                       reinterpret_cast<int32_t*>(base + w.experts), slots, rows, offsets, ws, w.base, s);
  if (st != UW_OK) return st;
  GroupedArgs a;
  a.N = gate->rows;
  a.K = gate->cols;
  a.E = gate->n_experts;
  a.swiglu = true;
  a.table[0] = gate->table;
  a.table[1] = up->table;
  a.x = x;
  a.x_rows = n_tokens;
  a.rows = rows;
  a.offsets = offsets;
  a.n_rows = n;
  a.y = base + w.h;
  a.ws = ws;
  a.ws_bytes = w.base;
  if ((st = launch_grouped(a, s)) != UW_OK) return st;
  GroupedArgs d;
  d.N = down->rows;
  d.K = down->cols;
  d.E = gate->n_experts;
  d.table[0] = down->table;
  d.x = reinterpret_cast<const uint16_t*>(base + w.h);
  d.x_rows = n;
  d.offsets = offsets;
  // the router finished before the gate/up product began to let this kernel
  // in, so the groups are known and the weights stream at once
  d.offsets_ready = true;
  d.n_rows = n;
  d.out_type = UW_OUT_FP32;  // each part is rounded once, after the weighted sum
  d.y = base + w.parts;
  d.ws = ws;
  d.ws_bytes = w.base;
  if ((st = launch_grouped(d, s)) != UW_OK) return st;
  return launch_combine(base + w.parts, UW_OUT_FP32, slots, weights, n_tokens, top_k, down->rows, n, residual, y, s);
}
