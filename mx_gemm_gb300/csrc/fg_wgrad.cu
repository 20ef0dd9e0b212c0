// Weights' gradients of products grouped by expert: out_e = A_e B_e^T for column
// operands A [N][P] and B [K][P] (fg_columns.cuh), the sum running over the places
// of expert e's slabs: out_e[n][k] = sum over its rows i of a[i][n] b[i][k].
//
// Both operands are e4m3 with one E8M0 per 32 places, which the tensor core applies
// itself, so a slab of 128 places is four block-scaled MMAs and nothing is folded
// by hand.  A pair of SMs takes 256 x 256 of the output at a time: each SM stages
// its own 128 rows of A and half of B's, and keeps its rows' 256 fp32 sums in
// tensor memory (cta_group::2).  Units run expert by expert, B's tiles innermost,
// so what the pairs take at one time shares its slabs in L2; an expert's slabs are
// 128 places, so nothing is gathered and nothing masked.  The last slab's MMAs end
// with its last 32 places that hold a row.
//
// What bounds it.  With s slabs an expert a unit is 4 s MMAs of 256 x 256 x 32 and
// 256 x 256 results to store: few rows an expert are bound by the output's bytes
// (HBM), many by the tensor cores.  The results leave their registers while the
// next unit's MMAs run: the accumulator is read whole, 128 registers a thread, and
// given back before anything is stored.  16 experts, 32768 rows, 4096 x 7168 to fp32:
// 652 us, 2.95 PFLOP/s, of which the results' 1.9 GB alone would take 277.
//
// An expert without rows has the gradient zero, which is stored (or, where the
// caller accumulates, left).
#include <cuda_bf16.h>

#include <atomic>
#include <cstring>

#include "fg_columns.cuh"
#include "fg_internal.cuh"
#include "fg_ptx.cuh"
#include "fg_tiles.cuh"

namespace fg {

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kPairThreads = 320;  // copies, MMAs, eight warps of results
constexpr int kStages = 6;
constexpr int kTmemCols = 512;
constexpr int kSum = 256;                    // columns of the sums
constexpr int kTile = kColumnSlab;           // bytes of 128 columns x 128 places
constexpr int kAtom = 512;
constexpr int kStage = (2 * kTile + 3 * kAtom + 1023) / 1024 * 1024;  // A, half of B, A's atom, B's two
constexpr int kScaleCols = 4 + 8;            // tensor memory of a stage's scales
static_assert(kSum + kStages * kScaleCols <= kTmemCols, "TMEM budget");

constexpr int smem_bytes(int E) { return kStages * kStage + 1024 + 8 * (E + 1); }
static_assert(smem_bytes(kMaxExperts) <= 232448 - 1024, "shared memory budget");

enum Output { kStoreF32, kAddF32, kStoreBf16 };

struct WgradParams {
  const int32_t* offsets;
  void* out;               // [E][N][K]
  uint32_t* err;
  uint64_t timeout_ns;
  int R, E, N, K, slabs;   // slabs: of the operands' rows
  int debug_stall;
};

// 256 x 256 of expert e's gradient; `slab0`: its first slab, `steps` of them, the
// last with `rest` rows.
struct WUnit {
  int e, nt, kt, slab0, steps, rest;
};

__device__ __forceinline__ void red_add2(float* p, float a, float b) {
  asm volatile("red.relaxed.gpu.global.add.v2.f32 [%0], {%1, %2};" ::"l"(p), "f"(a), "f"(b) : "memory");
}

// tmap_a, tmap_b: the operands' images as 2 KiB rows of 8-byte elements, boxes of a
// slab (8 rows); tmap_bh: B's, boxes of half a slab; tmap_asf, tmap_bsf: the atoms.
template <int OUT>
__global__ void __launch_bounds__(kPairThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                 const __grid_constant__ CUtensorMap tmap_bh, const __grid_constant__ CUtensorMap tmap_asf,
                 const __grid_constant__ CUtensorMap tmap_bsf, const WgradParams p) {
  extern __shared__ uint8_t dsmem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kStages];   // even SM: both SMs' copies of a stage landed
  __shared__ __align__(8) uint64_t empty_bar[kStages];  // both: the stage's MMAs are done
  __shared__ __align__(8) uint64_t accf_bar, acce_bar, stall_bar, drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, issued_sh, consumed_sh;
  int* offs_sh = reinterpret_cast<int*>(smem + kStages * kStage);  // clamped offsets [E + 1]
  int* slab_sh = offs_sh + p.E + 1;                                // slabs before each expert

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const uint64_t T = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    mbar_init(&accf_bar, 1);
    mbar_init(&acce_bar, 16);  // the eight result warps of each SM
    mbar_init(&stall_bar, 1);
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    issued_sh = 0;
    consumed_sh = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_base_sh, kTmemCols);
    tmem_relinquish_pair();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tmap_a);
    prefetch_tmap(&tmap_b);
    prefetch_tmap(&tmap_bh);
    prefetch_tmap(&tmap_asf);
    prefetch_tmap(&tmap_bsf);
  }
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  // the offsets as the quantiser of the operands reads them
  if (warp == 2) read_slabs(p.offsets, p.R, p.E, p.slabs, offs_sh, slab_sh);
  tc_fence_before();
  __syncthreads();
  // both SMs' barriers exist before either's copies or commits reach them
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  const int ntiles = p.N / 128, ktiles = p.K / 128;
  const int NT = (ntiles + 1) / 2, KT = (ktiles + 1) / 2;
  const long long units = static_cast<long long>(p.E) * NT * KT;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  auto unit = [&](long long u) {
    WUnit q;
    const int per = NT * KT;
    q.e = static_cast<int>(u / per);
    const int r = static_cast<int>(u - static_cast<long long>(q.e) * per);
    q.nt = r / KT;
    q.kt = r - q.nt * KT;
    q.slab0 = slab_sh[q.e];
    q.steps = slab_sh[q.e + 1] - q.slab0;
    q.rest = offs_sh[q.e + 1] - offs_sh[q.e] - (q.steps - 1) * kPlaces;
    q.e = __shfl_sync(0xffffffffu, q.e, 0);
    q.nt = __shfl_sync(0xffffffffu, q.nt, 0);
    q.kt = __shfl_sync(0xffffffffu, q.kt, 0);
    q.slab0 = __shfl_sync(0xffffffffu, q.slab0, 0);
    q.steps = __shfl_sync(0xffffffffu, q.steps, 0);
    q.rest = __shfl_sync(0xffffffffu, q.rest, 0);
    return q;
  };
  auto both = [&](const WUnit& q) { return 2 * q.kt + 1 < ktiles; };  // B has two tiles here
  // bytes that one SM's copies of a stage count
  auto stage_tx = [&](bool two) { return static_cast<uint32_t>(kTile + kAtom + (two ? kTile + 2 * kAtom : kTile / 2 + kAtom)); };

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    int it = 0;
    bool ok = true;
    for (long long u = pair; ok && u < units; u += pairs) {
      const WUnit q = unit(u);
      const bool two = both(q);
      const int at = min(2 * q.nt + rank, ntiles - 1) * p.slabs + q.slab0;      // this SM's slab of A
      const int b0 = 2 * q.kt * p.slabs + q.slab0, b1 = b0 + (two ? p.slabs : 0);  // B's tiles
      for (int i = 0; i < q.steps; ++i, ++it) {
        const int slot = it % kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[slot], ((it / kStages) & 1) ^ 1u, T, p.err, 81));
        if (!ok) break;
        uint8_t* st = smem + slot * kStage;
        const uint32_t fb = mapa_u32(&full_bar[slot], 0);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[slot], 2 * stage_tx(two));
          tma_load_2d_pair(st, &tmap_a, 0, (at + i) * 8, fb);
          if (two)
            tma_load_2d_pair(st + kTile, &tmap_b, 0, ((rank == 0 ? b0 : b1) + i) * 8, fb);
          else
            tma_load_2d_pair(st + kTile, &tmap_bh, 0, (b0 + i) * 8 + 4 * rank, fb);
          tma_load_2d_pair(st + 2 * kTile, &tmap_asf, 0, at + i, fb);
          tma_load_2d_pair(st + 2 * kTile + kAtom, &tmap_bsf, 0, b0 + i, fb);
          if (two) tma_load_2d_pair(st + 2 * kTile + 2 * kAtom, &tmap_bsf, 0, b1 + i, fb);
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      issued_sh = it;
      if (!ok) abort_sh = 1;
    }
  } else if (warp == 1) {
    // ----------------------------------------------------- MMAs (even SM only)
    if (rank == 0) {
      bool ok = true;
      if (p.debug_stall) ok = __all_sync(0xffffffffu, mbar_wait(&stall_bar, 0, T, p.err, 82));
      int it = 0, done = 0;  // done: units with rows so far
      for (long long u = pair; ok && u < units; u += pairs) {
        const WUnit q = unit(u);
        if (q.steps == 0) continue;
        ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar, (done & 1) ^ 1u, T, p.err, 83));
        if (!ok) break;
        ++done;
        tc_fence_after();
        const int width = both(q) ? 256 : 128;
        for (int i = 0; i < q.steps; ++i) {
          const int slot = it % kStages;
          ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[slot], (it / kStages) & 1, T, p.err, 84));
          if (!ok) break;
          ++it;  // this stage's copies have all landed
          tc_fence_after();
          const uint32_t st = smem_u32(smem) + slot * kStage;
          const uint32_t sfa = tmem + kSum + slot * kScaleCols, sfb = sfa + 4;
          const int parts = i + 1 < q.steps ? 4 : (q.rest + 31) / 32;  // blocks of 32 places with a row
          if (elect_one()) {
            const uint32_t sf = st + 2 * kTile;
            tc_cp_pair_32x128b_warpx4(sfa, sdesc_plain_rows16(sf));
            tc_cp_pair_32x128b_warpx4(sfb, sdesc_plain_rows16(sf + kAtom));
            if (width > 128) tc_cp_pair_32x128b_warpx4(sfb + 4, sdesc_plain_rows16(sf + 2 * kAtom));
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (j < parts)
                mma_mxf8f6f4_pair(tmem, sdesc_sw128(st + j * 32), sdesc_sw128(st + kTile + j * 32),
                                  idesc_mx(256, width, kF8f6f4E4M3, j, j), sfa, sfb, (i | j) != 0 ? 1u : 0u);
            tc_commit_pair_mc(&empty_bar[slot], 3);  // the stage is free again in both SMs
          }
          __syncwarp();
        }
        if (!ok) break;
        if (elect_one()) tc_commit_pair_mc(&accf_bar, 3);  // both SMs' rows are complete
        __syncwarp();
      }
      if (lane == 0) {
        consumed_sh = it;
        if (!ok) abort_sh = 1;
      }
      if (it > 0) {  // every MMA, copy and commit has landed before the teardown
        if (elect_one()) tc_commit_pair_mc(&drain_bar, 1);
        __syncwarp();
        mbar_wait(&drain_bar, 0, T, p.err, 85);
      }
    }
  } else {
    // -------------------------------------------------- results (both SMs)
    const int qd = warp & 3;
    const int c0 = ((warp - 2) >> 2) * 128;  // this warp's half of the columns
    int done = 0;
    for (long long u = pair; u < units; u += pairs) {
      const WUnit q = unit(u);
      if (q.steps == 0 && OUT == kAddF32) continue;
      // v[64 h + 32 c + 4 b + ..]: lanes 16 h .. + 15, columns 64 c + 8 b .. + 7 of this half
      uint32_t v[128];
      if (q.steps > 0) {
        const bool w = mbar_wait(&accf_bar, done & 1, T, p.err, 86);
        if (!__all_sync(0xffffffffu, w)) {
          if (lane == 0) abort_sh = 1;
          break;
        }
        ++done;
        tc_fence_after();
        const uint32_t taddr = tmem + c0 + (static_cast<uint32_t>(qd * 32) << 16);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < 2; ++c) tmem_ld_frag64(taddr + 64 * c + (static_cast<uint32_t>(16 * h) << 16), &v[64 * h + 32 * c]);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(&acce_bar, 0);  // the pair's next unit may overwrite the sums
      } else {
#pragma unroll
        for (int i = 0; i < 128; ++i) v[i] = 0u;
      }
      const int nt = 2 * q.nt + rank;
      const int k0 = q.kt * 256 + c0;
      if (nt >= ntiles || k0 >= p.K) continue;
      // A store covers eight rows x 32 bytes: whole sectors.
      const size_t row = (static_cast<size_t>(q.e) * p.N + nt * 128 + qd * 32 + (lane >> 2)) * p.K + k0;
      if (OUT == kStoreBf16) {
        // four lanes hold eight columns of two neighbouring blocks; the even ones
        // take four columns of the first each, the odd ones of the second
        __nv_bfloat16* out = static_cast<__nv_bfloat16*>(p.out) + row + ((lane & 2) << 1) + ((lane & 1) << 3);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < 16; b += 2) {
              const int x = 64 * h + 4 * b + 2 * r;
              const uint32_t first = pack_bf16x2(__uint_as_float(v[x]), __uint_as_float(v[x + 1]));
              const uint32_t second = pack_bf16x2(__uint_as_float(v[x + 4]), __uint_as_float(v[x + 5]));
              const uint32_t got = __shfl_xor_sync(0xffffffffu, lane & 1 ? first : second, 1);
              const uint2 o = lane & 1 ? make_uint2(got, second) : make_uint2(first, got);
              *reinterpret_cast<uint2*>(out + static_cast<size_t>(16 * h + 8 * r) * p.K + 8 * b) = o;
            }
      } else {
        float* out = static_cast<float*>(p.out) + row + 2 * (lane & 3);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int b = 0; b < 16; ++b) {
              const int x = 64 * h + 4 * b + 2 * r;
              float* to = out + static_cast<size_t>(16 * h + 8 * r) * p.K + 8 * b;
              if (OUT == kAddF32)
                red_add2(to, __uint_as_float(v[x]), __uint_as_float(v[x + 1]));
              else
                *reinterpret_cast<uint2*>(to) = make_uint2(v[x], v[x + 1]);
            }
      }
    }
  }

  // --------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // both SMs have stopped issuing; their counters are visible across the pair
  cluster_wait();
  if (rank == 0 && warp == 0) {
    const int peer_abort = static_cast<int>(ld_cluster_u32(mapa_u32(&abort_sh, 1)));
    if (abort_sh || peer_abort) {
      // Every stage phase that either SM's copies started must complete before
      // the pair's shared memory goes away: they count on these barriers.
      const int L = issued_sh;
      const int P = static_cast<int>(ld_cluster_u32(mapa_u32(&issued_sh, 1)));
      const int hi = L > P ? L : P;
      int first = 0;  // stages of the units before u
      for (long long u = pair; u < units && first < hi; u += pairs) {
        const WUnit q = unit(u);
        const uint32_t tx = stage_tx(both(q));
        if (lane == 0) {
          for (int it = max(first, consumed_sh); it < min(first + q.steps, hi); ++it) {
            const int slot = it % kStages;
            if (it >= L)
              mbar_arrive_expect_tx(&full_bar[slot], tx);  // only the odd SM issued this stage: arm it for its bytes
            else if (it >= P)
              mbar_complete_tx(&full_bar[slot], tx);  // the odd SM never issued its half of this stage
            mbar_wait(&full_bar[slot], (it / kStages) & 1, T, nullptr, 0);
          }
        }
        __syncwarp();
        first += q.steps;
      }
    }
  }
  __syncthreads();
  cluster_arrive();  // nothing is in flight towards either SM any more
  cluster_wait();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

void config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attrs)[2], int ctas, int E, cudaStream_t stream) {
  cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = smem_bytes(E);
  cfg.stream = stream;
  attrs[0].id = cudaLaunchAttributeClusterDimension;
  attrs[0].val.clusterDim.x = 2;
  attrs[0].val.clusterDim.y = 1;
  attrs[0].val.clusterDim.z = 1;
  attrs[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = pdl_enabled() ? 2 : 1;
}

// Pairs that the current device holds at once (looked up once; 0 on an error).
int wgrad_clusters() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (const int c = cached[dev].load(std::memory_order_relaxed)) return c;
  const void* kernel = reinterpret_cast<const void*>(&wgrad_kernel<kStoreF32>);
  if (ensure_smem_attr(kernel, smem_bytes(kMaxExperts)) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attrs[2];
  config(cfg, attrs, 512, kMaxExperts, nullptr);
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) return 0;
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

struct Maps {
  CUtensorMap a, b, bh, asf, bsf;
};

template <int OUT>
cudaError_t launch_out(const Maps& m, const WgradParams& p, int ctas, cudaStream_t stream) {
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&wgrad_kernel<OUT>), smem_bytes(kMaxExperts));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attrs[2];
  config(cfg, attrs, ctas, p.E, stream);
  return cudaLaunchKernelEx(&cfg, wgrad_kernel<OUT>, m.a, m.b, m.bh, m.asf, m.bsf, p);
}

}  // namespace

}  // namespace fg

using namespace fg;

extern "C" fg_status fg_grouped_wgrad(const fg_bshuf* a, const fg_bshuf* b, const int32_t* offsets, int64_t R, int E, int type,
                                      int accumulate, void* out, uint32_t flags, void* stream) {
  const char* what = "fg_grouped_wgrad";
  fg_status s = check_desc(a);
  if (s == FG_OK) s = check_desc(b);
  if (s != FG_OK) return s;
  if (a->mode != FG_MXFP8_B32 || b->mode != FG_MXFP8_B32)
    return fail(FG_ERR_LAYOUT, "%s: operands must be column operands (fg_quantize_columns)", what);
  if (flags & ~FG_FLAG_DEBUG_STALL) return fail(FG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
  if (type != FG_TYPE_F32 && type != FG_TYPE_BF16) return fail(FG_ERR_INVALID_ARG, "%s: bad type %d", what, type);
  if (accumulate && type != FG_TYPE_F32) return fail(FG_ERR_INVALID_ARG, "%s: sums are kept in fp32", what);
  const int64_t N = a->N, K = b->N;
  if ((s = check_columns(what, N, R, E)) != FG_OK) return s;
  if ((s = check_columns(what, K, R, E)) != FG_OK) return s;
  const int64_t slabs = column_slabs(R, E);
  if (a->K != slabs * kPlaces || b->K != slabs * kPlaces)
    return fail(FG_ERR_SHAPE, "%s: operands of %lld and %lld places, R=%lld rows of %d experts take %lld", what, (long long)a->K,
                (long long)b->K, (long long)R, E, (long long)(slabs * kPlaces));
  // the maps' coordinates, in rows of 2 KiB, are 32-bit
  if ((N / 128) * slabs * 8 > INT32_MAX || (K / 128) * slabs * 8 > INT32_MAX || N * K > (int64_t(1) << 40))
    return fail(FG_ERR_SHAPE, "%s: an operand is too large", what);
  if (!offsets || !out) return fail(FG_ERR_INVALID_ARG, "%s: null offsets or output", what);
  if (!aligned(offsets, 4) || !aligned(out, 16)) return fail(FG_ERR_ALIGN, "%s: offsets must be 4-byte aligned, the output 16-byte", what);
  if ((s = check_arch()) != FG_OK) return s;
  WgradParams p;
  memset(&p, 0, sizeof p);
  p.err = dev_error_ptr();
  if (!p.err) return fail(FG_ERR_CUDA, "device error word unavailable");
  Maps m;
  const int64_t arows = (N / 128) * slabs, brows = (K / 128) * slabs;
  if ((s = make_tmap_rows(&m.a, a->data, arows * 8, 2048, 8)) != FG_OK) return s;
  if ((s = make_tmap_rows(&m.b, b->data, brows * 8, 2048, 8)) != FG_OK) return s;
  if ((s = make_tmap_rows(&m.bh, b->data, brows * 8, 2048, 4)) != FG_OK) return s;
  if ((s = make_tmap_rows(&m.asf, a->sf, arows, 512, 1)) != FG_OK) return s;
  if ((s = make_tmap_rows(&m.bsf, b->sf, brows, 512, 1)) != FG_OK) return s;
  p.offsets = offsets;
  p.out = out;
  p.timeout_ns = wait_timeout_ns();
  p.R = static_cast<int>(R);
  p.E = E;
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.slabs = static_cast<int>(slabs);
  p.debug_stall = (flags & FG_FLAG_DEBUG_STALL) ? 1 : 0;
  const int64_t units = E * ((N / 128 + 1) / 2) * ((K / 128 + 1) / 2);
  const int most = wgrad_clusters();
  if (most == 0) return fail(FG_ERR_CUDA, "%s: no room for a pair of SMs", what);
  const int ctas = 2 * static_cast<int>(units < most ? units : most);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = type == FG_TYPE_BF16 ? launch_out<kStoreBf16>(m, p, ctas, st)
                        : accumulate         ? launch_out<kAddF32>(m, p, ctas, st)
                                             : launch_out<kStoreF32>(m, p, ctas, st);
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "weights' gradient launch");
}
