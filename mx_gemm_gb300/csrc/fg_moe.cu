// Routing of tokens to experts, and the weighted sum of the experts' rows:
// what stands before and after the products grouped by expert.
//
// Routing.  Per token the top_k largest of E logits (ties: the lowest expert;
// NaN counts as -infinity, and -infinity is never picked), their softmax, and
// the stable order of all (token, choice) pairs by expert: pair i = t * top_k +
// j goes to slot offsets[e] + (pairs before i with the same expert e).  A warp
// finds a token's choices in registers: logits as unsigned keys in the same
// order, top_k times the largest key (one warp reduction) and the lowest
// expert that has it (another).
//
// The stable order needs no sort, because a token picks an expert at most
// once: for 64 tokens at a time shared memory holds a 64-bit mask per expert,
// the warps set their tokens' bits (in any order: the result is the same), and
// a pair's rank is the expert's count so far plus the set bits below the
// token's own.  One block does up to 64 tokens alone (one launch).  More tokens
// are cut over the SMs: the first kernel leaves each pair's rank within its
// block's range and the block's counts, the second adds the counts of the
// blocks before it and scatters.
#include <cuda_bf16.h>

#include "fg_host.cuh"
#include "fg_internal.cuh"
#include "fg_ptx.cuh"

namespace fg {

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kGroup = 64;  // tokens whose picks one mask holds

struct RouteParams {
  const void* logits;
  float* weights;     // [T][k]
  int32_t* experts;   // [T][k]
  int32_t* offsets;   // [E + 1]
  int32_t* rows;      // [T * k]
  int32_t* slots;     // [T][k]
  uint32_t* counts;   // [blocks][E], more than one block only
  int64_t T, ldl;
  int E, k, renormalize;
};

__device__ __forceinline__ float ld_logit(const float* p) { return __ldcs(p); }
__device__ __forceinline__ float ld_logit(const __nv_bfloat16* p) {
  const unsigned short u = __ldcs(reinterpret_cast<const unsigned short*>(p));
  return __uint_as_float(static_cast<uint32_t>(u) << 16);
}

// Unsigned key in the order of the floats, both zeros alike; 0 for -infinity
// and NaN.
__device__ __forceinline__ uint32_t key_of(float l) {
  if (!(l > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(l + 0.f);  // -0 becomes +0
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}
// exp(l - top), 1 where both are infinite
__device__ __forceinline__ float exp_below(float l, float top) { return l == top ? 1.f : expf(l - top); }

// The choices of one token: lane j < k gets expert (-1: none left) and weight.
template <typename T, int VPL>
__device__ __forceinline__ void pick(const RouteParams& p, int64_t t, int lane, int& expert, float& weight) {
  const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
  uint32_t key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = i * 32 + lane;
    key[i] = e < p.E ? key_of(ld_logit(row + e)) : 0u;
  }
  // this lane's largest key and its first place
  uint32_t best = 0u;
  int at = 0;
  auto rescan = [&] {
    best = 0u;
    at = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (key[i] > best) {
        best = key[i];
        at = i;
      }
  };
  rescan();
  float top = 0.f, sum = 0.f;
  expert = -1;
  weight = 0.f;
  for (int j = 0; j < p.k; ++j) {
    const uint32_t m = __reduce_max_sync(0xffffffffu, best);
    if (m == 0u) break;  // no finite logit is left
    const int e = static_cast<int>(__reduce_min_sync(0xffffffffu, best == m ? static_cast<uint32_t>(at * 32 + lane) : ~0u));
    const float l = logit_of(m);
    if (j == 0) {
      top = l;
      if (!p.renormalize) {
        // over all experts, before any key is taken away
#pragma unroll
        for (int i = 0; i < VPL; ++i) sum += key[i] ? exp_below(logit_of(key[i]), top) : 0.f;
#pragma unroll
        for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
      }
    }
    const float w = exp_below(l, top);
    if (p.renormalize) sum += w;
    if (lane == j) {
      expert = e;
      weight = w;
    }
    if (lane == (e & 31)) {
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (i == at) key[i] = 0u;
      rescan();
    }
  }
  if (expert >= 0) weight = weight / sum;
}

// Exclusive sum of counts[0..E) into base[0..E], by the first warp.
__device__ __forceinline__ void scan_experts(const uint32_t* counts, uint32_t* base, int E) {
  if (threadIdx.x >= 32) return;
  const int lane = threadIdx.x;
  uint32_t carry = 0;
  for (int e0 = 0; e0 < E; e0 += 32) {
    const uint32_t c = e0 + lane < E ? counts[e0 + lane] : 0u;
    uint32_t s = c;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, s, d);
      if (lane >= d) s += o;
    }
    if (e0 + lane < E) base[e0 + lane] = carry + s - c;
    carry += __shfl_sync(0xffffffffu, s, 31);
  }
  if (lane == 0) base[E] = carry;
}

// Pairs [i0, i1): slot = base of the expert + rank, which slots[] holds so far.
__device__ __forceinline__ void scatter_pairs(const RouteParams& p, const uint32_t* base, int64_t i0, int64_t i1) {
  for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
    const int e = p.experts[i];
    if (e < 0) continue;
    const int32_t slot = static_cast<int32_t>(base[e]) + p.slots[i];
    p.slots[i] = slot;
    p.rows[slot] = static_cast<int32_t>(i / p.k);
  }
}

// Tokens [first, last) of block b of `blocks`.
__device__ __forceinline__ int64_t cut(int64_t T, int b, int blocks) { return T * b / blocks; }

// First kernel: choices, weights, ranks, and the block's counts.  Alone (one
// block) it also scans and scatters.
template <typename T, int VPL>
__global__ void __launch_bounds__(1024) route_kernel(const RouteParams p) {
  __shared__ uint32_t mask[kGroup / 32][kMaxExperts];
  __shared__ uint32_t count[kMaxExperts];
  __shared__ uint32_t base[kMaxExperts + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t first = cut(p.T, blockIdx.x, gridDim.x), last = cut(p.T, blockIdx.x + 1, gridDim.x);
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) count[e] = 0u;
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t0 = first; t0 < last; t0 += kGroup) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
#pragma unroll
      for (int w = 0; w < kGroup / 32; ++w) mask[w][e] = 0u;
    }
    __syncthreads();
    const int n = static_cast<int>(min(static_cast<int64_t>(kGroup), last - t0));
    for (int i = warp; i < n; i += warps) {
      int e;
      float w;
      pick<T, VPL>(p, t0 + i, lane, e, w);
      if (lane < p.k) {
        p.experts[(t0 + i) * p.k + lane] = e;
        p.weights[(t0 + i) * p.k + lane] = w;
        if (e >= 0) atomicOr(&mask[i >> 5][e], 1u << (i & 31));
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * p.k; i += blockDim.x) {
      const int e = p.experts[t0 * p.k + i];  // written by this block, before the barrier
      const int t = i / p.k;
      int32_t rank = -1;
      if (e >= 0) {
        rank = static_cast<int32_t>(count[e]);
#pragma unroll
        for (int w = 0; w < kGroup / 32; ++w) {
          const int below = t - 32 * w;  // tokens of this word before t
          const uint32_t m = below >= 32 ? ~0u : (below <= 0 ? 0u : (1u << below) - 1u);
          rank += __popc(mask[w][e] & m);
        }
      }
      p.slots[t0 * p.k + i] = rank;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
#pragma unroll
      for (int w = 0; w < kGroup / 32; ++w) count[e] += __popc(mask[w][e]);
    }
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x)
      p.counts[static_cast<size_t>(blockIdx.x) * p.E + e] = count[e];
    return;
  }
  scan_experts(count, base, p.E);
  __syncthreads();
  scatter_pairs(p, base, 0, p.T * p.k);
  for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = static_cast<int32_t>(base[e]);
  for (int64_t i = base[p.E] + threadIdx.x; i < p.T * p.k; i += blockDim.x) p.rows[i] = -1;
}

// Second kernel, over the same cuts of the tokens.
__global__ void __launch_bounds__(1024) route_scatter_kernel(const RouteParams p) {
  __shared__ uint32_t total[kMaxExperts];   // pairs of each expert
  __shared__ uint32_t before[kMaxExperts];  // ... in the blocks before this one
  __shared__ uint32_t base[kMaxExperts + 1];
  pdl_wait();
  pdl_launch_dependents();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    total[e] = 0u;
    before[e] = 0u;
  }
  __syncthreads();
  // threads in groups of E (rounded up to warps) share the blocks' counts
  const int width = (p.E + 31) / 32 * 32;
  const int groups = max(1, static_cast<int>(blockDim.x) / width);
  const int g = threadIdx.x / width;
  for (int e = threadIdx.x - g * width; e < p.E && g < groups; e += blockDim.x) {
    uint32_t all = 0, mine = 0;
    for (int b = g; b < static_cast<int>(gridDim.x); b += groups) {
      const uint32_t c = p.counts[static_cast<size_t>(b) * p.E + e];
      all += c;
      if (b < static_cast<int>(blockIdx.x)) mine += c;
    }
    atomicAdd(&total[e], all);
    atomicAdd(&before[e], mine);
  }
  __syncthreads();
  scan_experts(total, base, p.E);
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = threadIdx.x; e <= p.E; e += blockDim.x) p.offsets[e] = static_cast<int32_t>(base[e]);
  }
  const int64_t pairs = p.T * p.k;
  const int64_t routed = base[p.E];
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) base[e] += before[e];
  __syncthreads();
  scatter_pairs(p, base, cut(p.T, blockIdx.x, gridDim.x) * p.k, cut(p.T, blockIdx.x + 1, gridDim.x) * p.k);
  for (int64_t i = routed + static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < pairs;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    p.rows[i] = -1;
}

int route_blocks(int64_t T) {
  if (T <= kGroup) return 1;
  const int64_t n = (T + kGroup - 1) / kGroup;
  return static_cast<int>(n < sm_count() ? n : sm_count());
}

template <typename T>
cudaError_t launch_route(const RouteParams& p, cudaStream_t st) {
  const int blocks = route_blocks(p.T);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  // a warp per token, and threads enough for the experts' loops
  const int64_t warps = p.T < 8 ? 8 : (p.T < 32 ? p.T : 32);
  cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  const int vpl = (p.E + 31) / 32;
  cudaError_t e;
  if (vpl <= 1) e = cudaLaunchKernelEx(&cfg, route_kernel<T, 1>, p);
  else if (vpl <= 2) e = cudaLaunchKernelEx(&cfg, route_kernel<T, 2>, p);
  else if (vpl <= 4) e = cudaLaunchKernelEx(&cfg, route_kernel<T, 4>, p);
  else if (vpl <= 8) e = cudaLaunchKernelEx(&cfg, route_kernel<T, 8>, p);
  else if (vpl <= 16) e = cudaLaunchKernelEx(&cfg, route_kernel<T, 16>, p);
  else e = cudaLaunchKernelEx(&cfg, route_kernel<T, 32>, p);
  if (e != cudaSuccess || blocks == 1) return e;
  return cudaLaunchKernelEx(&cfg, route_scatter_kernel, p);
}

// ------------------------------------------------------------------ combine

constexpr int kVec = 8;      // bf16 values per thread
constexpr int kUnroll = 8;   // experts' rows in flight per thread

__device__ __forceinline__ void fma8(float (&acc)[kVec], const uint4& u, float w) {
  const uint32_t q[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    acc[2 * i] = fmaf(w, __uint_as_float(q[i] << 16), acc[2 * i]);
    acc[2 * i + 1] = fmaf(w, __uint_as_float(q[i] & 0xffff0000u), acc[2 * i + 1]);
  }
}

// out[t] = residual[t] + sum_j weights[t][j] * Y[slots[t][j]], in the order of
// j, 32-bit sums; slots outside [0, R) count as no choice.  One thread per
// token and eight columns; HBM-bound: every chosen row is read once.
__global__ void __launch_bounds__(128) combine_kernel(const __nv_bfloat16* __restrict__ Y, int64_t R,
                                                      const int32_t* __restrict__ slots,
                                                      const float* __restrict__ weights, const __nv_bfloat16* residual,
                                                      int k, int64_t N, __nv_bfloat16* out) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t t = blockIdx.x;
  const int64_t c = (static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x) * kVec;
  if (c >= N) return;
  float acc[kVec] = {};
  if (residual) fma8(acc, __ldcs(reinterpret_cast<const uint4*>(residual + t * N + c)), 1.f);
  for (int j0 = 0; j0 < k; j0 += kUnroll) {
    uint4 v[kUnroll];
    float w[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      w[j] = 0.f;
      if (j0 + j < k) {
        const int64_t s = __ldg(slots + t * k + j0 + j);
        if (s >= 0 && s < R) {
          w[j] = __ldg(weights + t * k + j0 + j);
          v[j] = __ldcs(reinterpret_cast<const uint4*>(Y + s * N + c));
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) fma8(acc, v[j], w[j]);
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[2 * i], acc[2 * i + 1]);
    o[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(out + t * N + c) = make_uint4(o[0], o[1], o[2], o[3]);
}

}  // namespace

}  // namespace fg

using namespace fg;

extern "C" {

fg_status fg_moe_route_workspace_size(int64_t T, int E, uint64_t* bytes) {
  if (!bytes) return fail(FG_ERR_INVALID_ARG, "null output");
  if (T < 0 || E < 1 || E > kMaxExperts)
    return fail(FG_ERR_SHAPE, "fg_moe_route: T=%lld, E=%d (1..%d experts)", (long long)T, E, kMaxExperts);
  const int blocks = route_blocks(T);
  *bytes = blocks > 1 ? static_cast<uint64_t>(blocks) * E * 4 : 0;
  return FG_OK;
}

fg_status fg_moe_route(const void* logits, int type, int64_t T, int E, int64_t ldl, int top_k, uint32_t flags,
                       float* weights, int32_t* experts, int32_t* offsets, int32_t* rows, int32_t* slots,
                       void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* what = "fg_moe_route";
  if (type != FG_TYPE_F32 && type != FG_TYPE_BF16) return fail(FG_ERR_INVALID_ARG, "%s: bad type %d", what, type);
  if (flags & ~FG_FLAG_RENORMALIZE) return fail(FG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
  uint64_t need = 0;
  fg_status s = fg_moe_route_workspace_size(T, E, &need);
  if (s != FG_OK) return s;
  if (top_k < 1 || top_k > kMaxTopK || top_k > E)
    return fail(FG_ERR_SHAPE, "%s: top_k=%d outside 1..min(%d, E=%d)", what, top_k, kMaxTopK, E);
  if (T * top_k > (int64_t(1) << 30)) return fail(FG_ERR_SHAPE, "%s: T=%lld too large", what, (long long)T);
  if (ldl < E) return fail(FG_ERR_SHAPE, "%s: logit rows %lld apart, shorter than E=%d", what, (long long)ldl, E);
  if (!offsets || (T > 0 && (!logits || !weights || !experts || !rows || !slots)))
    return fail(FG_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned(logits, type == FG_TYPE_F32 ? 4 : 2) || !aligned(weights, 4) || !aligned(experts, 4) ||
      !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(workspace, 4))
    return fail(FG_ERR_ALIGN, "%s: a pointer is not aligned to its type", what);
  if (need && (!workspace || workspace_bytes < need))
    return fail(FG_ERR_WORKSPACE, "%s: T=%lld, E=%d need a %llu-byte workspace", what, (long long)T, E,
                (unsigned long long)need);
  if ((s = check_arch()) != FG_OK) return s;
  RouteParams p{logits, weights, experts, offsets, rows, slots, static_cast<uint32_t*>(workspace),
                T, ldl, E, top_k, (flags & FG_FLAG_RENORMALIZE) ? 1 : 0};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == FG_TYPE_F32 ? launch_route<float>(p, st) : launch_route<__nv_bfloat16>(p, st);
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "routing launch");
}

fg_status fg_moe_combine(const void* Y, int64_t R, const int32_t* slots, const float* weights, const void* residual,
                         int64_t T, int top_k, int64_t N, void* out, void* stream) {
  const char* what = "fg_moe_combine";
  if (T < 0 || R < 0 || N <= 0 || N % kVec)
    return fail(FG_ERR_SHAPE, "%s: T=%lld, R=%lld, N=%lld (N a positive multiple of 8)", what, (long long)T, (long long)R,
                (long long)N);
  if (top_k < 1 || top_k > kMaxTopK) return fail(FG_ERR_SHAPE, "%s: top_k=%d outside 1..%d", what, top_k, kMaxTopK);
  if (T > (int64_t(1) << 30) || N > (int64_t(1) << 24)) return fail(FG_ERR_SHAPE, "%s: T or N too large", what);
  if (T == 0) return FG_OK;
  if ((R > 0 && !Y) || !slots || !weights || !out) return fail(FG_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned(Y, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(slots, 4) || !aligned(weights, 4))
    return fail(FG_ERR_ALIGN, "%s: Y, residual and out must be 16-byte aligned, slots and weights 4-byte", what);
  fg_status s = check_arch();
  if (s != FG_OK) return s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(T), static_cast<unsigned>((N / kVec + 127) / 128));
  cfg.blockDim = dim3(128);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, combine_kernel, static_cast<const __nv_bfloat16*>(Y), R, slots, weights,
                                           static_cast<const __nv_bfloat16*>(residual), top_k, N,
                                           static_cast<__nv_bfloat16*>(out));
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "combine launch");
}

}  // extern "C"
