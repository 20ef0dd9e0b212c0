// Routing of tokens to experts, and the weighted sum of the experts' rows:
// what stands before and after the products grouped by expert.
//
// Routing.  Per token the top_k largest of E logits (ties: the lowest expert;
// NaN counts as -infinity, and -infinity is never picked), their softmax, and
// the stable order of all (token, choice) pairs by expert: pair i = t * top_k +
// j goes to slot offsets[e] + (pairs before i with the same expert e).  A warp
// finds a token's choices in registers: logits as unsigned keys in the same
// order with the expert's complement below them, so that one comparison also
// breaks ties.  Each lane sorts its own few keys once (Batcher's odd-even
// merge; up to 256 experts); then top_k times the warp takes the largest head
// (one reduction for 16-bit logits, two for 32-bit ones) and its lane moves up.
// Against scanning the lane's keys anew for each choice this took 16383 x 256
// from 29 us to 11 for this kernel (16.5 us with the second, where 10 MB of HBM
// would take 1.6): it is bound by instructions, 475 a token and warp.  One token
// is bound by the call: 7 us of host time, 2 to 3 of them the launch.
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
#include "fg_logits.cuh"
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
  uint32_t* counts;   // [blocks][E rounded up to 4], more than one block only
  int64_t T, ldl;
  int E, k, renormalize;
  int whole;  // rows of logits are aligned to a lane's chunk
};

// Sortable form of a logit and its expert: the larger comes first, among equal
// logits the lower expert; 0 for -infinity and NaN, which are never picked.
// Both zeros have one key.
template <typename T>
struct Key;

template <>
struct Key<float> {
  using Word = unsigned long long;  // key, complement of the expert
  static __device__ __forceinline__ Word make(uint32_t bits, int e) {
    const float l = __uint_as_float(bits) + 0.f;  // -0 becomes +0
    const int32_t u = __float_as_int(l);
    const uint32_t k = static_cast<uint32_t>(u ^ ((u >> 31) | 0x80000000));  // negative: complement; else: sign set
    return l > -INFINITY ? (static_cast<Word>(k) << 32) | static_cast<uint32_t>(~e) : 0ull;
  }
  static __device__ __forceinline__ Word largest(Word w) {
    const uint32_t hi = static_cast<uint32_t>(w >> 32);
    const uint32_t m = __reduce_max_sync(0xffffffffu, hi);
    const uint32_t lo = __reduce_max_sync(0xffffffffu, hi == m ? static_cast<uint32_t>(w) : 0u);
    return (static_cast<Word>(m) << 32) | lo;
  }
  static __device__ __forceinline__ int expert(Word w) { return ~static_cast<int>(w); }
  static __device__ __forceinline__ float logit(Word w) {
    const uint32_t k = static_cast<uint32_t>(w >> 32);
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
  }
};

template <>
struct Key<__nv_bfloat16> {
  using Word = uint32_t;  // key in the upper half, complement of the expert in the lower
  static __device__ __forceinline__ Word make(uint32_t bits, int e) {
    const float l = __uint_as_float(bits << 16) + 0.f;  // -0 becomes +0
    const int32_t u = __float_as_int(l);
    const uint32_t k = static_cast<uint32_t>(u ^ ((u >> 31) | 0x80000000));  // negative: complement; else: sign set
    return l > -INFINITY ? (k & 0xffff0000u) | (0xffffu - e) : 0u;
  }
  static __device__ __forceinline__ Word largest(Word w) { return __reduce_max_sync(0xffffffffu, w); }
  static __device__ __forceinline__ int expert(Word w) { return 0xffff - static_cast<int>(w & 0xffffu); }
  static __device__ __forceinline__ float logit(Word w) {
    const uint32_t k = w >> 16;
    return __uint_as_float(((k & 0x8000u) ? (k & 0x7fffu) : (k ^ 0xffffu)) << 16);
  }
};

// Batcher's odd-even merge sort, largest first, all indexes known at compile time.
template <int N, typename W>
__device__ __forceinline__ void sort_down(W (&a)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2) {
#pragma unroll
    for (int k = p; k >= 1; k /= 2) {
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k) {
#pragma unroll
        for (int i = 0; i < k; ++i) {
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const W x = a[i + j], y = a[i + j + k];
            a[i + j] = x > y ? x : y;
            a[i + j + k] = x > y ? y : x;
          }
        }
      }
    }
  }
}

// The choices of one token: lane j < k gets expert (-1: none left) and weight.
template <typename T, int VPL>
__device__ __forceinline__ void pick(const RouteParams& p, const Logits<T, VPL>& l, int lane, int& expert, float& weight) {
  using K = Key<T>;
  typename K::Word key[VPL];
#pragma unroll
  for (int i = 0; i < VPL; ++i) key[i] = K::make(l.bits[i], Logits<T, VPL>::expert(i, lane));
  // the lane's largest key: first of the sorted ones; with more than eight the
  // network outgrows the registers, and the lane that gave one looks again
  constexpr bool SORTED = VPL <= 8;
  typename K::Word head = 0;
  auto look = [&] {
    head = key[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) head = key[i] > head ? key[i] : head;
  };
  if constexpr (SORTED) {
    sort_down(key);
    head = key[0];
  } else {
    look();
  }
  const typename K::Word first = K::largest(head);
  float sum = 0.f;
  if (!p.renormalize) {  // over all experts, before any key is taken away
#pragma unroll
    for (int i = 0; i < VPL; ++i) sum += key[i] ? exp_below(K::logit(key[i]), K::logit(first)) : 0.f;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  }
  // the lane whose head was taken moves up; once none is left m stays 0
  typename K::Word mine = lane == 0 ? first : 0, m = first;
  if (SORTED && p.k <= 8) {
    // written out: a step needs no more of the sorted keys than choices are left
#pragma unroll
    for (int j = 1; j < 8; ++j) {
      if (j >= p.k) break;
      const bool taken = key[0] == m;  // one lane: experts differ
#pragma unroll
      for (int i = 0; i < 8 - j && i < VPL; ++i) key[i] = taken ? (i + 1 < VPL ? key[i + 1 < VPL ? i + 1 : 0] : 0) : key[i];
      m = K::largest(key[0]);
      mine = lane == j ? m : mine;
    }
  } else {
#pragma unroll 1
    for (int j = 1; j < p.k; ++j) {
      if (head == m) {
        if constexpr (SORTED) {
#pragma unroll
          for (int i = 0; i + 1 < VPL; ++i) key[i] = key[i + 1];
          key[VPL - 1] = 0;
          head = key[0];
        } else {
#pragma unroll
          for (int i = 0; i < VPL; ++i) key[i] = key[i] == m ? 0 : key[i];
          look();
        }
      }
      m = K::largest(head);
      mine = lane == j ? m : mine;
    }
  }
  expert = mine ? K::expert(mine) : -1;
  weight = mine ? exp_below(K::logit(mine), K::logit(first)) : 0.f;
  if (p.renormalize) {
    sum = weight;
#pragma unroll
    for (int d = 16; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  }
  if (mine) weight = weight / sum;
}

// Exclusive sum of counts[0..E) into base[0..E], by the whole block; ends with
// the block in step.
__device__ __forceinline__ void scan_experts(const uint32_t* counts, uint32_t* base, int E) {
  __shared__ uint32_t part[kMaxExperts / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int chunks = (E + 31) / 32;
  for (int c = warp; c < chunks; c += warps) {
    const int e = c * 32 + lane;
    const uint32_t n = e < E ? counts[e] : 0u;
    uint32_t sum = n;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const uint32_t o = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += o;
    }
    if (e < E) base[e] = sum - n;
    if (lane == 31) part[c] = sum;
  }
  __syncthreads();
  for (int c = warp; c < chunks; c += warps) {
    const int e = c * 32 + lane;
    const uint32_t below = __reduce_add_sync(0xffffffffu, lane < c ? part[lane] : 0u);
    if (e < E) base[e] += below;
    if (c == chunks - 1 && lane == 0) base[E] = below + part[c];
  }
  __syncthreads();
}

// Pairs [i0, i1): slot = base of the expert + rank, which slots[] holds so far.
__device__ __forceinline__ void scatter_pairs(const RouteParams& p, const uint32_t* base, int64_t i0, int64_t i1) {
  for (int64_t i = i0 + threadIdx.x; i < i1; i += blockDim.x) {
    const int e = p.experts[i];
    if (e < 0) continue;
    const int32_t slot = static_cast<int32_t>(base[e]) + p.slots[i];
    p.slots[i] = slot;
    p.rows[slot] = static_cast<int32_t>(static_cast<uint32_t>(i) / static_cast<uint32_t>(p.k));  // i < 2^30
  }
}

// Tokens [first, last) of block b of `blocks`.
__device__ __forceinline__ int64_t cut(int64_t T, int b, int blocks) { return T * b / blocks; }

// First kernel: choices, weights, ranks, and the block's counts.  Alone (one
// block) it also scans and scatters.  Blocks of 1024 threads have 64 registers
// each; where a lane sorts more than eight keys they are 512 threads wide.
constexpr int route_threads(int vpl) { return vpl <= 8 ? 1024 : 512; }

template <typename T, int VPL>
__global__ void __launch_bounds__(route_threads(VPL)) route_kernel(const RouteParams p) {
  // tokens of a group that a warp takes: the launch has a warp for each token
  // or route_threads / 32
  constexpr int TPW = kGroup * 32 / route_threads(VPL);
  __shared__ uint32_t mask[kGroup / 32][kMaxExperts];
  __shared__ uint32_t count[kMaxExperts];
  __shared__ uint32_t base[kMaxExperts + 1];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int64_t first = cut(p.T, blockIdx.x, gridDim.x), last = cut(p.T, blockIdx.x + 1, gridDim.x);
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
    count[e] = 0u;
#pragma unroll
    for (int w = 0; w < kGroup / 32; ++w) mask[w][e] = 0u;
  }
  pdl_wait();
  pdl_launch_dependents();
  for (int64_t t0 = first; t0 < last; t0 += kGroup) {
    const int n = static_cast<int>(min(static_cast<int64_t>(kGroup), last - t0));
    Logits<T, VPL> next;
    if (warp < n) next.load(p, t0 + warp, lane);
    __syncthreads();
    int expert[TPW];
#pragma unroll
    for (int h = 0; h < TPW; ++h) {
      const int i = warp + h * warps;
      expert[h] = -1;
      if (i < n) {
        const Logits<T, VPL> now = next;
        if (h + 1 < TPW && i + warps < n) next.load(p, t0 + i + warps, lane);  // on its way during this token's work
        float w;
        pick<T, VPL>(p, now, lane, expert[h], w);
        if (lane < p.k) {
          p.experts[(t0 + i) * p.k + lane] = expert[h];
          p.weights[(t0 + i) * p.k + lane] = w;
          if (expert[h] >= 0) atomicOr(&mask[i >> 5][expert[h]], 1u << (i & 31));
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int h = 0; h < TPW; ++h) {
      const int i = warp + h * warps;
      if (i < n && lane < p.k) {
        const int e = expert[h];
        int32_t rank = -1;
        if (e >= 0) {
          // the expert's pairs of earlier groups, of earlier words, and before i in its own
          rank = static_cast<int32_t>(count[e]) + __popc(mask[i >> 5][e] & ((1u << (i & 31)) - 1u));
#pragma unroll
          for (int w = 0; w + 1 < kGroup / 32; ++w) rank += i >= 32 * (w + 1) ? __popc(mask[w][e]) : 0;
        }
        p.slots[(t0 + i) * p.k + lane] = rank;
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
#pragma unroll
      for (int w = 0; w < kGroup / 32; ++w) {
        count[e] += __popc(mask[w][e]);
        mask[w][e] = 0u;
      }
    }
  }
  __syncthreads();
  if (gridDim.x > 1) {
    for (int e = threadIdx.x; e < p.E; e += blockDim.x)
      p.counts[static_cast<size_t>(blockIdx.x) * ((p.E + 3) & ~3) + e] = count[e];
    return;
  }
  scan_experts(count, base, p.E);
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
  // every block reads all counts, four experts a thread, the blocks' rows
  // shared out over the threads
  const int quads = (p.E + 3) / 4;
  const int groups = static_cast<int>(blockDim.x) / quads;  // E <= 1024: at least 4
  const int g = threadIdx.x / quads, e4 = (threadIdx.x - g * quads) * 4;
  if (g < groups) {
    uint32_t all[4] = {}, mine[4] = {};
    const uint4* row = reinterpret_cast<const uint4*>(p.counts) + e4 / 4;
    const int blocks = gridDim.x;
    for (int b0 = g; b0 < blocks; b0 += 4 * groups) {
      uint4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int b = b0 + i * groups;
        v[i] = b < blocks ? __ldcg(row + static_cast<size_t>(b) * quads) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        const bool before_me = b0 + i * groups < static_cast<int>(blockIdx.x);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          all[j] += c[j];
          mine[j] += before_me ? c[j] : 0u;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (e4 + j < p.E) {  // (the row's padding is not counted)
        atomicAdd(&total[e4 + j], all[j]);
        atomicAdd(&before[e4 + j], mine[j]);
      }
    }
  }
  __syncthreads();
  scan_experts(total, base, p.E);
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
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  auto launch = [&](auto kernel, int most) {
    // a warp per token, and threads enough for the experts' loops
    const int64_t warps = p.T < 8 ? 8 : (p.T < most / 32 ? p.T : most / 32);
    cfg.blockDim = dim3(static_cast<unsigned>(32 * warps));
    return cudaLaunchKernelEx(&cfg, kernel, p);
  };
  const int vpl = (p.E + 31) / 32;
  cudaError_t e;
  if (vpl <= 1) e = launch(route_kernel<T, 1>, route_threads(1));
  else if (vpl <= 2) e = launch(route_kernel<T, 2>, route_threads(2));
  else if (vpl <= 4) e = launch(route_kernel<T, 4>, route_threads(4));
  else if (vpl <= 8) e = launch(route_kernel<T, 8>, route_threads(8));
  else if (vpl <= 16) e = launch(route_kernel<T, 16>, route_threads(16));
  else e = launch(route_kernel<T, 32>, route_threads(32));
  if (e != cudaSuccess || blocks == 1) return e;
  cfg.blockDim = dim3(1024);
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
// token and eight columns, its top_k rows' loads in flight together.  HBM-bound:
// every chosen row is read once; 8191 tokens x 8 rows of 7168 in 168 us (7.0
// TB/s with 5 % of the tokens padding, at the rate of a copy).
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
  if (T < 0 || T > (int64_t(1) << 30) || E < 1 || E > kMaxExperts)
    return fail(FG_ERR_SHAPE, "fg_moe_route: T=%lld, E=%d (1..%d experts)", (long long)T, E, kMaxExperts);
  const int blocks = route_blocks(T);
  *bytes = blocks > 1 ? static_cast<uint64_t>(blocks) * ((E + 3) / 4 * 4) * 4 : 0;
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
  if (T > (int64_t(1) << 30) / top_k) return fail(FG_ERR_SHAPE, "%s: T=%lld too large", what, (long long)T);
  if (ldl < E) return fail(FG_ERR_SHAPE, "%s: logit rows %lld apart, shorter than E=%d", what, (long long)ldl, E);
  if (!offsets || (T > 0 && (!logits || !weights || !experts || !rows || !slots)))
    return fail(FG_ERR_INVALID_ARG, "%s: null pointer", what);
  if (!aligned(logits, type == FG_TYPE_F32 ? 4 : 2) || !aligned(weights, 4) || !aligned(experts, 4) ||
      !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(slots, 4))
    return fail(FG_ERR_ALIGN, "%s: a pointer is not aligned to its type", what);
  if (need && !aligned(workspace, 16)) return fail(FG_ERR_ALIGN, "%s: workspace must be 16-byte aligned", what);
  if (need && (!workspace || workspace_bytes < need))
    return fail(FG_ERR_WORKSPACE, "%s: T=%lld, E=%d need a %llu-byte workspace", what, (long long)T, E,
                (unsigned long long)need);
  if ((s = check_arch()) != FG_OK) return s;
  RouteParams p{logits, weights, experts, offsets, rows, slots, static_cast<uint32_t*>(workspace),
                T, ldl, E, top_k, (flags & FG_FLAG_RENORMALIZE) ? 1 : 0, 0};
  // a lane's chunk: at most 16 bytes, and no more than its share of the experts
  const int es = type == FG_TYPE_F32 ? 4 : 2;
  int vpl = 1;
  while (vpl < (E + 31) / 32) vpl *= 2;
  const int chunk = vpl * es < 16 ? vpl * es : 16;
  p.whole = aligned(logits, chunk) && (T <= 1 || ldl * es % chunk == 0) ? 1 : 0;
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
