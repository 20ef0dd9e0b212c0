// The router's side of a training step: the balance loss with the counts that it
// weighs, and the gradient of the logits.
//
// With p = softmax(l_t) (0 in rows with nothing to pick: NaN counts as -infinity),
// T' the tokens with something to pick and f_e expert e's share of all choices:
//   P_e = sum_t p_te / T',  loss = c E sum_e f_e P_e,  slope_e = c E f_e / T',
// the loss's derivative by each token's p_te (f is piecewise constant).  The
// gradient of a token's logits from the slopes and from those of its routing
// weights, dw_j:
//   dl_e = p_e (slope_e - sum_i p_i slope_i) + q_j (dw_j - sum_i q_i dw_i)   [e = expert j]
// where q is the softmax over the chosen ones; with weights that are shares of all
// experts q_j = p_j and the last sum is subtracted from every p_e instead.
//
// A warp takes a token, its logits in registers.  The sums over tokens stay in
// registers to the end of a warp's tokens, go over shared memory in the order of
// the warps, and over the blocks' partials in theirs: the same call gives the same
// bits.  Both are bound by instructions and by their start, not by HBM: 16383 x 256 bf16
// in 10 us with the counts (balance and its sums; 14 with the blocks' sums joined by one
// block) and 9.0 us (gradient), where the bytes take 1.2 and 2.5.  A token takes some 400
// and 550 instructions of a warp, 8 exponentials among them.
#include <cuda_bf16.h>

#include <type_traits>

#include "fg_host.cuh"
#include "fg_internal.cuh"
#include "fg_logits.cuh"
#include "fg_ptx.cuh"

namespace fg {

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;

struct BalanceParams {
  const void* logits;
  const int32_t* offsets;  // [E + 1]
  float* part;             // [blocks][E + 2]: sums of p, tokens, sums x counts (more than one block only)
  float* loss;             // [1]
  int32_t* counts;         // [E]
  float* probs;            // [E]
  float* slopes;           // [E]
  int64_t T, ldl;
  float coefficient;
  int E, whole;
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) v += __shfl_xor_sync(0xffffffffu, v, d);
  return v;
}

// N sums over the warp, their steps next to one another.
template <int N>
__device__ __forceinline__ void warp_sums(float (&v)[N]) {
#pragma unroll
  for (int d = 16; d > 0; d /= 2) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], d);
  }
}

__device__ __forceinline__ float warp_max(float v) {
  float m;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
  return m;
}

// exp(l - top) of a lane's logits (0 for -infinity and NaN) and the largest, `top`
// (-infinity: nothing to pick; +infinity: the infinite ones share alike).
template <typename T, int VPL>
__device__ __forceinline__ float exponentials(const Logits<T, VPL>& l, float (&p)[VPL]) {
  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    p[i] = fmaxf(__uint_as_float(sizeof(T) == 2 ? l.bits[i] << 16 : l.bits[i]), -INFINITY);  // (a NaN is not kept)
    top = fmaxf(top, p[i]);
  }
  top = warp_max(top);
  if (fabsf(top) < INFINITY) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = expf(p[i] - top);
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) p[i] = top > 0.f && p[i] == top ? 1.f : 0.f;
  }
  return top;
}

__device__ __forceinline__ int count_of(const BalanceParams& p, int e) {
  return max(__ldg(p.offsets + e + 1) - __ldg(p.offsets + e), 0);
}

// Sums over the blocks' rows of [E + 2] that everything is divided by, for the whole
// block: choices, tokens, and the counts' products with the sums of p.
struct Totals {
  float per_choice, per_token, dot;
};

__device__ __forceinline__ Totals totals(const BalanceParams& p, const float* part, int blocks) {
  __shared__ int count_sh[32];
  __shared__ float sums_sh[2];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int stride = p.E + 2;
  int mine = 0;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) mine += count_of(p, e);
  if (warp == 0) {
    // (tokens: whole numbers up to 2^24, exact)
    float s[2] = {0.f, 0.f};
#pragma unroll 8
    for (int b = lane; b < blocks; b += 32) {
      s[0] += part[static_cast<size_t>(b) * stride + p.E];
      s[1] += part[static_cast<size_t>(b) * stride + p.E + 1];
    }
    warp_sums(s);
    if (lane == 0) {
      sums_sh[0] = s[0];
      sums_sh[1] = s[1];
    }
  }
  mine = __reduce_add_sync(0xffffffffu, mine);
  if (lane == 0) count_sh[warp] = mine;
  __syncthreads();
  const int all = __reduce_add_sync(0xffffffffu, lane < warps ? count_sh[lane] : 0);
  Totals t;
  t.per_choice = all > 0 ? 1.f / static_cast<float>(all) : 0.f;
  t.per_token = sums_sh[0] > 0.f ? 1.f / sums_sh[0] : 0.f;
  t.dot = sums_sh[1];
  return t;
}

// Expert e's outputs from the sum of its p over all tokens; expert 0's thread has the loss.
__device__ __forceinline__ void put(const BalanceParams& p, const Totals& t, int e, float sum) {
  const int n = count_of(p, e);
  const float c = p.coefficient * static_cast<float>(p.E);
  p.probs[e] = sum * t.per_token;
  p.counts[e] = n;
  p.slopes[e] = c * (static_cast<float>(n) * t.per_choice) * t.per_token;
  if (e == 0) *p.loss = c * (t.dot * t.per_choice * t.per_token);
}

// Warps of a block at most: with 32 a thread has 64 registers, which sums of more
// than eight experts a lane outgrow.
constexpr int balance_warps(int vpl) { return vpl <= 8 ? 32 : (vpl <= 16 ? 16 : 8); }

// Blocks' sums of p, tokens, and the sums' product with the counts, so that the loss
// needs no sum over experts later; alone (one block) also the rest.  Dynamic shared
// memory: [warps][E + 2].
template <typename T, int VPL>
__global__ void __launch_bounds__(32 * balance_warps(VPL)) balance_kernel(const BalanceParams p) {
  extern __shared__ float sums_sh[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int stride = p.E + 2;
  pdl_wait();
  pdl_launch_dependents();
  float acc[VPL] = {};
  int tokens = 0;
  const int64_t step = static_cast<int64_t>(gridDim.x) * warps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp;
  Logits<T, VPL> next;
  if (t < p.T) next.load(p, t, lane);
  for (; t < p.T; t += step) {
    const Logits<T, VPL> now = next;
    if (t + step < p.T) next.load(p, t + step, lane);  // on its way during this token's work
    float v[VPL], sum = 0.f;
    tokens += exponentials(now, v) > -INFINITY;
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += v[i];
    sum = warp_sum(sum);
    const float r = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < VPL; ++i) acc[i] = fmaf(v[i], r, acc[i]);
  }
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = Logits<T, VPL>::expert(i, lane);
    if (e < p.E) sums_sh[warp * stride + e] = acc[i];
  }
  if (lane == 0) sums_sh[warp * stride + p.E] = static_cast<float>(tokens);
  __syncthreads();
  float* to = gridDim.x > 1 ? p.part + static_cast<size_t>(blockIdx.x) * stride : sums_sh;
  float dot = 0.f;
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) {
    float s = 0.f;
#pragma unroll 8
    for (int w = 0; w < warps; ++w) s += sums_sh[w * stride + e];
    to[e] = s;
    if (e < p.E) dot = fmaf(static_cast<float>(count_of(p, e)), s, dot);
  }
  __shared__ float dot_sh[32];
  dot = warp_sum(dot);
  if (lane == 0) dot_sh[warp] = dot;
  __syncthreads();
  if (warp == 0) {
    dot = warp_sum(lane < warps ? dot_sh[lane] : 0.f);
    if (lane == 0) to[p.E + 1] = dot;
  }
  if (gridDim.x > 1) return;
  __syncthreads();
  const Totals all = totals(p, sums_sh, 1);
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) put(p, all, e, sums_sh[e]);
}

// 32 experts a block, the blocks' rows shared out over its 32 warps.
__global__ void __launch_bounds__(1024) balance_finish_kernel(const BalanceParams p, int blocks) {
  __shared__ float sum_sh[32][33];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int stride = p.E + 2, e = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (e < p.E) {
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) s += p.part[static_cast<size_t>(b) * stride + e];
  }
  sum_sh[warp][lane] = s;
  const Totals all = totals(p, p.part, blocks);  // (the block is in step after it)
  if (warp == 0 && e < p.E) {
    s = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) s += sum_sh[w][lane];
    put(p, all, e, s);
  }
}

// ----------------------------------------------------------- logits' gradient

constexpr int kBackwardWarps = 8;

struct BackwardParams {
  const void* logits;
  const int32_t* experts;  // [T][k] (dweights given)
  const float* dweights;   // [T][k] or null
  const float* slopes;     // [E] or null
  void* out;               // [T][E]
  int64_t T, ldl;
  int E, k, renormalize, whole, whole_out;
};

// Shared memory: a row of values for each warp, zero between tokens.
template <typename T, int VPL>
__global__ void __launch_bounds__(32 * kBackwardWarps) route_backward_kernel(const BackwardParams p) {
  using L = Logits<T, VPL>;
  __shared__ __align__(16) float rows_sh[kBackwardWarps][32 * VPL];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  float* row = rows_sh[warp];
  for (int e = lane; e < 32 * VPL; e += 32) row[e] = 0.f;
  __syncwarp();
  pdl_wait();
  pdl_launch_dependents();
  float slope[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = L::expert(i, lane);
    slope[i] = p.slopes && e < p.E ? __ldg(p.slopes + e) : 0.f;
  }
  const int64_t step = static_cast<int64_t>(gridDim.x) * warps;
  int64_t t = static_cast<int64_t>(blockIdx.x) * warps + warp;
  L next;
  if (t < p.T) next.load(p, t, lane);
  for (; t < p.T; t += step) {
    const L now = next;
    int expert = -1;
    float dw = 0.f, chosen = -INFINITY;
    if (p.dweights && lane < p.k) {
      expert = __ldg(p.experts + t * p.k + lane);
      dw = __ldg(p.dweights + t * p.k + lane);
      if (expert >= p.E) expert = -1;
      if (expert >= 0) {
        const T* l = static_cast<const T*>(p.logits) + t * p.ldl + expert;
        chosen = static_cast<float>(*l);
      }
    }
    if (t + step < p.T) next.load(p, t + step, lane);
    float v[VPL];
    const float top = exponentials(now, v);
    chosen = fmaxf(chosen, -INFINITY);  // (a NaN is not kept)
    // what lies beside no choice need not be a number that q = 0 could be multiplied with
    dw = chosen > -INFINITY ? dw : 0.f;
    // sums of the exponentials, of their products with the slopes, and of the chosen
    // ones' and theirs with dweights
    float q = chosen > -INFINITY ? exp_below(chosen, top) : 0.f;
    float sums[4] = {0.f, 0.f, q, q * dw};
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      sums[0] += v[i];
      sums[1] = fmaf(v[i], slope[i], sums[1]);
    }
    warp_sums(sums);
    // Choices that routing would not make may lie so far below the token's largest logit
    // that all of theirs are 0: renormalised, they are taken by their own largest.
    if (p.renormalize && p.dweights && sums[2] < 0.0625f) {
      const float own = warp_max(chosen);
      q = chosen > -INFINITY ? exp_below(chosen, own) : 0.f;
      float s[2] = {q, q * dw};
      warp_sums(s);
      sums[2] = s[0];
      sums[3] = s[1];
    }
    const float r = sums[0] > 0.f ? 1.f / sums[0] : 0.f;
    const float share = p.renormalize ? (sums[2] > 0.f ? 1.f / sums[2] : 0.f) : r;
    const float mean = sums[3] * share;
    const float dot = fmaf(sums[1], r, p.renormalize ? 0.f : mean);
    if (p.dweights) {
      float add = q * share * (p.renormalize ? dw - mean : dw);
      // an expert that a token names twice (routing never does) takes both, in their order
      const unsigned peers = __match_any_sync(0xffffffffu, expert);
      const bool twice = expert >= 0 && (peers & (peers - 1)) != 0;
      if (__any_sync(0xffffffffu, twice)) {
        float sum = 0.f;
        for (int j = 0; j < 32; ++j) {
          const float other = __shfl_sync(0xffffffffu, add, j);
          if ((peers >> j) & 1u) sum += other;
        }
        add = sum;
      }
      if (expert >= 0) row[expert] = add;
      __syncwarp();
    }
    T* out = static_cast<T*>(p.out) + t * p.E;
#pragma unroll
    for (int c = 0; c < VPL; c += L::V) {
      const int e0 = L::expert(c, lane);
      alignas(16) float d[L::V];
      if constexpr (L::V % 4 == 0) {
#pragma unroll
        for (int i = 0; i < L::V; i += 4) *reinterpret_cast<float4*>(&d[i]) = *reinterpret_cast<const float4*>(row + e0 + i);
      } else {
#pragma unroll
        for (int i = 0; i < L::V; ++i) d[i] = row[e0 + i];
      }
#pragma unroll
      for (int i = 0; i < L::V; ++i) {
        d[i] = fmaf(v[c + i] * r, slope[c + i] - dot, d[i]);
      }
      if (p.whole_out && e0 + L::V <= p.E) {
        constexpr int BYTES = L::V * sizeof(T);
        alignas(16) T o[L::V];
#pragma unroll
        for (int i = 0; i < L::V; ++i) o[i] = static_cast<T>(d[i]);
        if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(out + e0) = *reinterpret_cast<const uint4*>(o);
        else if constexpr (BYTES == 8) *reinterpret_cast<uint2*>(out + e0) = *reinterpret_cast<const uint2*>(o);
        else if constexpr (BYTES == 4) *reinterpret_cast<uint32_t*>(out + e0) = *reinterpret_cast<const uint32_t*>(o);
        else out[e0] = o[0];
      } else {
#pragma unroll
        for (int i = 0; i < L::V; ++i)
          if (e0 + i < p.E) out[e0 + i] = static_cast<T>(d[i]);
      }
    }
    __syncwarp();
    if (expert >= 0) row[expert] = 0.f;
    __syncwarp();
  }
}

// ------------------------------------------------------------------- launch

void config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& attr, int64_t blocks, int threads, int smem, cudaStream_t st) {
  cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
}

// Calls f with the kernel for a lane's share of E experts.
template <typename F>
cudaError_t by_share(int E, F f) {
  const int vpl = (E + 31) / 32;
  if (vpl <= 1) return f(std::integral_constant<int, 1>());
  if (vpl <= 2) return f(std::integral_constant<int, 2>());
  if (vpl <= 4) return f(std::integral_constant<int, 4>());
  if (vpl <= 8) return f(std::integral_constant<int, 8>());
  if (vpl <= 16) return f(std::integral_constant<int, 16>());
  return f(std::integral_constant<int, 32>());
}

// Warps of a block of the balance loss for E experts (their rows fit 33 KB).
int warps_of_balance(int E) { return E <= 256 ? balance_warps(8) : (E <= 512 ? balance_warps(16) : balance_warps(32)); }

// One block alone up to four tokens a warp, else up to one an SM.
int balance_blocks(int64_t T, int E) {
  const int warps = warps_of_balance(E);
  if (T <= 4 * warps) return 1;
  const int64_t want = (T + 2 * warps - 1) / (2 * warps), most = sm_count();
  return static_cast<int>(want < most ? want : most);
}

// Whether rows of logits can be read a lane's chunk at a time (see Logits).
int whole_rows(const void* p, int type, int64_t T, int E, int64_t ld) {
  const int es = type == FG_TYPE_F32 ? 4 : 2;
  int vpl = 1;
  while (vpl < (E + 31) / 32) vpl *= 2;
  const int chunk = vpl * es < 16 ? vpl * es : 16;
  return aligned(p, chunk) && (T <= 1 || ld * es % chunk == 0) ? 1 : 0;
}

fg_status check_logits(const char* what, const void* logits, int type, int64_t T, int E, int64_t ldl) {
  if (type != FG_TYPE_F32 && type != FG_TYPE_BF16) return fail(FG_ERR_INVALID_ARG, "%s: bad type %d", what, type);
  if (T < 0 || T > (int64_t(1) << 24) || E < 1 || E > kMaxExperts)
    return fail(FG_ERR_SHAPE, "%s: T=%lld (up to 2^24), E=%d (1..%d experts)", what, (long long)T, E, kMaxExperts);
  if (T == 0) return FG_OK;
  if (ldl < E) return fail(FG_ERR_SHAPE, "%s: logit rows %lld apart, shorter than E=%d", what, (long long)ldl, E);
  if (!logits) return fail(FG_ERR_INVALID_ARG, "%s: null logits", what);
  if (!aligned(logits, type == FG_TYPE_F32 ? 4 : 2)) return fail(FG_ERR_ALIGN, "%s: logits are not aligned to their type", what);
  return FG_OK;
}

}  // namespace

}  // namespace fg

using namespace fg;

extern "C" {

fg_status fg_moe_balance_loss_workspace_size(int64_t T, int E, uint64_t* bytes) {
  if (!bytes) return fail(FG_ERR_INVALID_ARG, "null output");
  if (T < 0 || T > (int64_t(1) << 24) || E < 1 || E > kMaxExperts)
    return fail(FG_ERR_SHAPE, "fg_moe_balance_loss: T=%lld (up to 2^24), E=%d (1..%d experts)", (long long)T, E, kMaxExperts);
  const int blocks = balance_blocks(T, E);
  *bytes = blocks > 1 ? static_cast<uint64_t>(blocks) * (E + 2) * 4 : 0;
  return FG_OK;
}

fg_status fg_moe_balance_loss(const void* logits, int type, int64_t T, int E, int64_t ldl, const int32_t* offsets,
                              float coefficient, float* loss, int32_t* counts, float* probs, float* slopes,
                              void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* what = "fg_moe_balance_loss";
  fg_status s = check_logits(what, logits, type, T, E, ldl);
  if (s != FG_OK) return s;
  if (!offsets || !loss || !counts || !probs || !slopes) return fail(FG_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned(offsets, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(probs, 4) || !aligned(slopes, 4))
    return fail(FG_ERR_ALIGN, "%s: a pointer is not aligned to its type", what);
  uint64_t need = 0;
  if ((s = fg_moe_balance_loss_workspace_size(T, E, &need)) != FG_OK) return s;
  if (need && (!workspace || workspace_bytes < need))
    return fail(FG_ERR_WORKSPACE, "%s: T=%lld, E=%d need a %llu-byte workspace", what, (long long)T, E, (unsigned long long)need);
  if (need && !aligned(workspace, 4)) return fail(FG_ERR_ALIGN, "%s: workspace must be 4-byte aligned", what);
  if ((s = check_arch()) != FG_OK) return s;
  BalanceParams p{logits, offsets, static_cast<float*>(workspace), loss, counts, probs, slopes, T, ldl, coefficient, E,
                  whole_rows(logits, type, T, E, ldl)};
  const int blocks = balance_blocks(T, E);
  int warps = warps_of_balance(E);
  if (T < warps) warps = T < 4 ? 4 : static_cast<int>(T);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  config(cfg, attr, blocks, 32 * warps, warps * (E + 2) * 4, static_cast<cudaStream_t>(stream));
  cudaError_t e = by_share(E, [&](auto share) {
    constexpr int VPL = decltype(share)::value;
    return type == FG_TYPE_F32 ? cudaLaunchKernelEx(&cfg, balance_kernel<float, VPL>, p)
                               : cudaLaunchKernelEx(&cfg, balance_kernel<__nv_bfloat16, VPL>, p);
  });
  if (e == cudaSuccess && blocks > 1) {
    config(cfg, attr, (E + 31) / 32, 1024, 0, static_cast<cudaStream_t>(stream));
    e = cudaLaunchKernelEx(&cfg, balance_finish_kernel, p, blocks);
  }
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "balance loss launch");
}

fg_status fg_moe_route_backward(const void* logits, int type, int64_t T, int E, int64_t ldl, const int32_t* experts,
                                const float* dweights, int top_k, const float* slopes, uint32_t flags, void* out,
                                void* stream) {
  const char* what = "fg_moe_route_backward";
  if (flags & ~FG_FLAG_RENORMALIZE) return fail(FG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
  fg_status s = check_logits(what, logits, type, T, E, ldl);
  if (s != FG_OK) return s;
  if (dweights && (top_k < 1 || top_k > kMaxTopK || top_k > E))
    return fail(FG_ERR_SHAPE, "%s: top_k=%d outside 1..min(%d, E=%d)", what, top_k, kMaxTopK, E);
  if (T == 0) return FG_OK;
  if (!out || (dweights && !experts)) return fail(FG_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned(out, type == FG_TYPE_F32 ? 4 : 2) || !aligned(experts, 4) || !aligned(dweights, 4) || !aligned(slopes, 4))
    return fail(FG_ERR_ALIGN, "%s: a pointer is not aligned to its type", what);
  if ((s = check_arch()) != FG_OK) return s;
  BackwardParams p{logits, experts, dweights, slopes, out, T, ldl, E, top_k, (flags & FG_FLAG_RENORMALIZE) ? 1 : 0,
                   whole_rows(logits, type, T, E, ldl), whole_rows(out, type, T, E, E)};
  // four blocks an SM (16383 x 256, without choices' own largest logit: 8.7 us; two 10.2,
  // eight 9.8; 16384 x 512: 13.8, 12.7, 15.9)
  const int64_t want = (T + kBackwardWarps - 1) / kBackwardWarps, most = 4 * static_cast<int64_t>(sm_count());
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  config(cfg, attr, want < most ? want : most, 32 * kBackwardWarps, 0, static_cast<cudaStream_t>(stream));
  const cudaError_t e = by_share(E, [&](auto share) {
    constexpr int VPL = decltype(share)::value;
    return type == FG_TYPE_F32 ? cudaLaunchKernelEx(&cfg, route_backward_kernel<float, VPL>, p)
                               : cudaLaunchKernelEx(&cfg, route_backward_kernel<__nv_bfloat16, VPL>, p);
  });
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "logits' gradient launch");
}

}  // extern "C"
