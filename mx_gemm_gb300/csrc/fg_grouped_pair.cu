// Products grouped by expert on pairs of SMs: token tiles of up to 256 rows
// against two weight tiles at a time.  Schedule and layouts as in fg_grouped.cu.
//
// Why pairs.  One SM's tile of 128 weight rows x n tokens moves, per K step,
// 16 KB of weights and n * 128 bytes of tokens into shared memory and the MMA
// reads both again: at n = 208 that is 86 KB through a 128-byte port, 670
// cycles, while the tensor core needs 410.  On a pair the tokens are staged
// half by each SM and the hardware hands each half to both (cta_group::2), so
// an SM moves 58 KB: 450 cycles.  Measured, 64 experts, 4096 x 7168, 32768 rows
// that lie in place, unevenly routed (the whole call): mxfp4 438 us one-SM, 333 now
// (5.8 PFLOP/s; 293 where all experts have as many rows); 32-K mxfp8 795, 659 (2.9);
// fp8 x fp4 749, 606; bf16 (32 experts, 16384 rows) 725, 617 (1.6, at the power limit).
// Rows gathered by index cost their layout on top: mxfp4 375 to 385 us.  A
// step takes 520 (bf16) to 640 (mxfp4) cycles, the tensor pipe busy for 430 of
// them; the rest is the issue of the scale copies and the barriers.  With 64 rows
// an expert the weights' bytes bound it: mxfp8 301 us, 6.65 TB/s.
//
// Tried and dropped: tiles of 192 rows with two accumulators (mxfp4 436 us: more
// steps of the same length), a second copying warp (no faster), prefetches of the
// weights to L2 (356 -> 393 us), asking for the next barrier a step ahead (equal).
//
// The even SM's warp 1 issues the MMAs (256 weight rows x n tokens; rows
// 0..127 accumulate in the even SM's tensor memory, 128..255 in the odd one's);
// both SMs' copies count on the even one's barriers, and its commits free the
// stage in both.  The weight's scales are needed per SM, the tokens' for all n
// in both.  The other roles are those of the one-SM kernel.
//
// Where an expert's weight tiles are odd in number the last pair's odd SM
// computes the even one's tile again and stores nothing.
#include <cuda_bf16.h>

#include <atomic>

#include "fg_grouped.cuh"
#include "fg_ptx.cuh"
#include "fg_tiles.cuh"

namespace fg {

namespace {

constexpr int TT = 256;
constexpr int kPairThreads = 320;  // copies, MMAs, eight warps of results
constexpr int kTmemCols = 512;

template <int MODE>
struct PCfg {
  static constexpr int APS = MODE == kMXFP4 ? 2 : (is_mx(MODE) ? 1 : 0);
  static constexpr int STAGES = 6;
  static constexpr int TOK_BYTES = TT / 2 * 128;  // this SM's half of the tile
  static constexpr int W_TX = MODE == kMXFP4FP8A ? kSlabBytes / 2 : kSlabBytes;
  static constexpr int SFW_BYTES = APS * 512;
  static constexpr int SFT_BYTES = 2 * APS * 512;
  static constexpr int STAGE_RAW = kSlabBytes + TOK_BYTES + SFW_BYTES + SFT_BYTES;
  static constexpr int STAGE_BYTES = (STAGE_RAW + 1023) / 1024 * 1024;
  static constexpr int SFW_COLS = APS * 4, SFT_COLS = APS * 8;
  static constexpr int OUT_BYTES = 8 * 512;  // per result warp: 8 rows of Y x 32 columns
  static constexpr int smem(int E) { return STAGES * STAGE_BYTES + OUT_BYTES + 1024 + 8 * (E + 1); }
  static_assert(STAGES * STAGE_BYTES + OUT_BYTES + 1024 + 8 * (kMaxExperts + 1) <= 232448 - 1024, "shared memory budget");
  static_assert(TT + STAGES * (SFW_COLS + SFT_COLS) <= kTmemCols, "TMEM budget");
};

template <int MODE>
__device__ __forceinline__ void mma_step_pair(uint32_t d, uint64_t a, uint64_t b, int n, int j, int kb, uint32_t sfw,
                                              uint32_t sft, uint32_t accum) {
  if (MODE == kBF16) {
    mma_f16_pair(d, a, b, idesc_bf16(256, n), accum);
  } else if (MODE == kTensor) {
    mma_f8f6f4_pair(d, a, b, idesc_e4m3(256, n), accum);
  } else if (MODE == kMXFP8) {  // byte kb % 4 of the four-slab atoms
    mma_mxf8f6f4_pair(d, a, b, idesc_mx(256, n, kF8f6f4E4M3, kb & 3, kb & 3), sfw, sft, accum);
  } else if (MODE == kMXFP8B32) {
    mma_mxf8f6f4_pair(d, a, b, idesc_mx(256, n, kF8f6f4E4M3, j, j), sfw, sft, accum);
  } else if (MODE == kMXFP4FP8A) {
    mma_mxf8f6f4_pair(d, a, b, idesc_mx_ab(256, n, kF8f6f4E2M1, kF8f6f4E4M3, j, j), sfw, sft, accum);
  } else {
    const int g = j >> 1, id = 2 * (j & 1);
    mma_mxf4_pair(d, a, b, idesc_mx(256, n, kMxf4E2M1, id, id), sfw + 4 * g, sft + 8 * g, accum);
  }
}

template <int MODE>
__global__ void __launch_bounds__(kPairThreads, 1)
    grouped_pair_kernel(const __grid_constant__ AMaps a_maps, const __grid_constant__ CUtensorMap tmap_w,
                        const __grid_constant__ CUtensorMap tmap_wsf, const __grid_constant__ CUtensorMap tmap_asf,
                        const GroupedParams p) {
  using C = PCfg<MODE>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t dsmem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[ST];   // even SM: both SMs' copies of a stage landed
  __shared__ __align__(8) uint64_t empty_bar[ST];  // both: the stage's MMAs are done
  __shared__ __align__(8) uint64_t accf_bar, acce_bar, stall_bar, drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, issued_sh, consumed_sh;
  int* offs_sh = reinterpret_cast<int*>(smem + ST * C::STAGE_BYTES + C::OUT_BYTES);
  int* tiles_sh = offs_sh + p.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const uint64_t T = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
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
    for (int i = 0; i < 8; ++i) prefetch_tmap(&a_maps.rows[i]);
    prefetch_tmap(&tmap_w);
    if (C::APS) {
      prefetch_tmap(&tmap_wsf);
      prefetch_tmap(&tmap_asf);
    }
  }
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  read_offsets<TT>(p.offsets, p.R, p.E, offs_sh, tiles_sh);
  tc_fence_before();
  __syncthreads();
  // both SMs' barriers exist before either's copies or commits reach them
  cluster_arrive();
  cluster_wait();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  const int wtiles = p.N / 128;  // weight tiles of an expert
  Schedule s;
  s.offs = offs_sh;
  s.tiles = tiles_sh;
  s.E = p.E;
  s.NT = (wtiles + 1) / 2;
  s.KB = p.KB;
  s.units = static_cast<long long>(tiles_sh[p.E]) * s.NT;
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);
  const int shares = pair < s.units ? static_cast<int>((s.units - pair + pairs - 1) / pairs) : 0;
  auto unit = [&](int i) { return uniform(unit_at<TT>(s, pair + static_cast<long long>(i) * pairs)); };
  // bytes that one SM's copies of a stage of unit q count
  auto stage_tx = [&](const Unit& q) {
    return static_cast<uint32_t>(C::W_TX + q.width * 64 + C::SFW_BYTES + C::SFT_BYTES);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    int it = 0;
    bool ok = true;
    for (int i = 0; ok && i < shares; ++i) {
      const Unit q = unit(i);
      const int wt = q.e * wtiles + min(2 * q.nt + rank, wtiles - 1);  // this SM's tile of the stacked image
      const int half = q.width >> 1, row0 = q.row0 + rank * half;      // its rows of the token tile
      const CUtensorMap* a_map = &a_maps.rows[half / 16 - 1];
      for (int kb = 0; kb < s.KB; ++kb, ++it) {
        const int slot = it % ST;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[slot], ((it / ST) & 1) ^ 1u, T, p.err, 71));
        if (!ok) break;
        uint8_t* st = smem + slot * C::STAGE_BYTES;
        const uint32_t fb = mapa_u32(&full_bar[slot], 0);
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(&full_bar[slot], 2 * stage_tx(q));
          if (MODE == kMXFP4FP8A)
            tma_load_3d_pair(st, &tmap_w, 0, 0, wt * s.KB + kb, fb);
          else
            tma_load_2d_pair(st, &tmap_w, 0, (wt * s.KB + kb) * 8, fb);
          uint8_t* tok = st + kSlabBytes;
          tma_load_2d_pair(tok, a_map, kb * 128, row0, fb);
          if (C::APS) {
            const int watom = MODE == kMXFP8 ? wt * ((s.KB + 3) / 4) + kb / 4 : (wt * s.KB + kb) * C::APS;
            const int tatom = MODE == kMXFP8 ? q.tile * ((s.KB + 3) / 4) + kb / 4 : (q.tile * s.KB + kb) * C::APS;
            tma_load_2d_pair(tok + C::TOK_BYTES, &tmap_wsf, 0, watom, fb);
            tma_load_2d_pair(tok + C::TOK_BYTES + C::SFW_BYTES, &tmap_asf, 0, 2 * tatom, fb);
          }
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
      if (p.debug_stall) ok = __all_sync(0xffffffffu, mbar_wait(&stall_bar, 0, T, p.err, 72));
      int it = 0;
      for (int i = 0; ok && i < shares; ++i) {
        const Unit q = unit(i);
        ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar, (i & 1) ^ 1u, T, p.err, 73));
        if (!ok) break;
        tc_fence_after();
        for (int kb = 0; kb < s.KB; ++kb) {
          const int slot = it % ST;
          ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[slot], (it / ST) & 1, T, p.err, 74));
          if (!ok) break;
          ++it;  // this stage's copies have all landed
          tc_fence_after();
          const uint32_t st = smem_u32(smem) + slot * C::STAGE_BYTES;
          const uint32_t sfw = tmem + TT + slot * (C::SFW_COLS + C::SFT_COLS);
          const uint32_t sft = sfw + C::SFW_COLS;
          if (elect_one()) {
            if (C::APS) {
              const uint32_t sw = st + kSlabBytes + C::TOK_BYTES;
              const uint32_t stk = sw + C::SFW_BYTES;
#pragma unroll
              for (int g = 0; g < C::APS; ++g) {
                tc_cp_pair_32x128b_warpx4(sfw + 4 * g, sdesc_plain_rows16(sw + 512 * g));
                tc_cp_pair_32x128b_warpx4(sft + 8 * g, sdesc_plain_rows16(stk + 1024 * g));
                if (q.width > 128) tc_cp_pair_32x128b_warpx4(sft + 8 * g + 4, sdesc_plain_rows16(stk + 1024 * g + 512));
              }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_step_pair<MODE>(tmem, sdesc_sw128(st + j * 32), sdesc_sw128(st + kSlabBytes + j * 32), q.width, j, kb, sfw,
                                  sft, (kb | j) != 0 ? 1u : 0u);
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
        mbar_wait(&drain_bar, 0, T, p.err, 75);
      }
    }
  } else {
    // -------------------------------------------------- results (both SMs)
    const int qd = warp & 3;
    const int m0 = ((warp - 2) >> 2) * 128;  // this warp's half of the tile's rows
    uint8_t* stg_ptr = smem + ST * C::STAGE_BYTES + (warp - 2) * 512;
    const uint32_t stg = smem_u32(stg_ptr);
    const float scale = MODE == kTensor ? __ldg(static_cast<const float*>(p.a_scales)) * __ldg(p.b_s) : 1.f;
    for (int i = 0; i < shares; ++i) {
      const Unit q = unit(i);
      const bool w = mbar_wait(&accf_bar, i & 1, T, p.err, 76);
      if (!__all_sync(0xffffffffu, w)) {
        if (lane == 0) abort_sh = 1;
        break;
      }
      tc_fence_after();
      // v[64 h + 32 c + ..]: lanes 16 h .. 16 h + 15 (weight rows), columns 64 c .. (tokens)
      uint32_t v[128];
      const uint32_t taddr = tmem + m0 + (static_cast<uint32_t>(qd * 32) << 16);
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int c = 0; c < 2; ++c) tmem_ld_frag64(taddr + 64 * c + (static_cast<uint32_t>(16 * h) << 16), &v[64 * h + 32 * c]);
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(&acce_bar, 0);  // the pair's next tile may overwrite the accumulator
      const int nt = 2 * q.nt + rank;
      if (nt >= wtiles) continue;
      // Eight rows of Y at a time: the fragments go through shared memory
      // transposed, 64 bytes a row (16-byte piece i of row j at i ^ (j / 2 % 4)),
      // and leave as 16-byte stores.  (Storing each lane's weight row two bytes
      // at a time took 9000 cycles a tile, longer than the MMAs of K = 2048.)
      __nv_bfloat16* out = p.y + static_cast<size_t>(q.row0 + m0 + (lane >> 2)) * p.N + nt * 128 + qd * 32 + (lane & 3) * 8;
      const uint32_t put = stg + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
      const uint4* get = reinterpret_cast<const uint4*>(stg_ptr + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4));
#pragma unroll
      for (int b = 0; b < 16; ++b) {
        if (m0 + 8 * b >= q.count) break;
        const int k = 32 * (b >> 3) + 4 * (b & 7);
        auto pack = [&](int x) { return pack_bf16x2(__uint_as_float(v[x]) * scale, __uint_as_float(v[x + 1]) * scale); };
        stmatrix4_trans(put, pack(k), pack(k + 2), pack(64 + k), pack(64 + k + 2));
        __syncwarp();
        const uint4 o = *get;
        __syncwarp();
        if (m0 + 8 * b + (lane >> 2) < q.count) *reinterpret_cast<uint4*>(out + static_cast<size_t>(8 * b) * p.N) = o;
      }
    }
  }

  // --------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  cluster_arrive();  // both SMs have stopped issuing; their counters are visible across the pair
  cluster_wait();
  if (rank == 0 && threadIdx.x == 0) {
    const int peer_abort = static_cast<int>(ld_cluster_u32(mapa_u32(&abort_sh, 1)));
    if (abort_sh || peer_abort) {
      // Every stage phase that either SM's copies started must complete before
      // the pair's shared memory goes away: they count on these barriers.
      const int L = issued_sh;
      const int P = static_cast<int>(ld_cluster_u32(mapa_u32(&issued_sh, 1)));
      const int hi = L > P ? L : P;
      for (int it = consumed_sh; it < hi; ++it) {
        const int slot = it % ST;
        const uint32_t tx = stage_tx(unit_at<TT>(s, pair + static_cast<long long>(it / s.KB) * pairs));
        if (it >= L)
          mbar_arrive_expect_tx(&full_bar[slot], tx);  // only the odd SM issued this stage: arm it for its bytes
        else if (it >= P)
          mbar_complete_tx(&full_bar[slot], tx);  // the odd SM never issued its half of this stage
        mbar_wait(&full_bar[slot], (it / ST) & 1, T, nullptr, 0);
      }
    }
  }
  __syncthreads();
  cluster_arrive();  // nothing is in flight towards either SM any more
  cluster_wait();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_pair(tmem, kTmemCols);
}

template <int MODE>
void config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attrs)[2], int ctas, int E, cudaStream_t stream) {
  cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = PCfg<MODE>::smem(E);
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

template <int MODE>
cudaError_t launch_mode(const AMaps& a_maps, const CUtensorMap& tmap_w, const CUtensorMap& tmap_wsf,
                        const CUtensorMap& tmap_asf, const GroupedParams& p, int ctas, cudaStream_t stream) {
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&grouped_pair_kernel<MODE>), PCfg<MODE>::smem(kMaxExperts));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attrs[2];
  config<MODE>(cfg, attrs, ctas, p.E, stream);
  return cudaLaunchKernelEx(&cfg, grouped_pair_kernel<MODE>, a_maps, tmap_w, tmap_wsf, tmap_asf, p);
}

}  // namespace

// Pairs that the current device holds at once (looked up once; 0 on an error).
int grouped_pair_clusters() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  if (const int c = cached[dev].load(std::memory_order_relaxed)) return c;
  constexpr int MODE = kMXFP4;  // the largest footprint
  if (ensure_smem_attr(reinterpret_cast<const void*>(&grouped_pair_kernel<MODE>), PCfg<MODE>::smem(kMaxExperts)) != cudaSuccess)
    return 0;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attrs[2];
  config<MODE>(cfg, attrs, 512, kMaxExperts, nullptr);
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, reinterpret_cast<const void*>(&grouped_pair_kernel<MODE>), &cfg) != cudaSuccess || n <= 0)
    return 0;
  cached[dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_grouped_pair(int mode, const AMaps& a_maps, const CUtensorMap& tmap_w, const CUtensorMap& tmap_wsf,
                                const CUtensorMap& tmap_asf, const GroupedParams& p, int ctas, cudaStream_t stream) {
  switch (mode) {
    case kBF16: return launch_mode<kBF16>(a_maps, tmap_w, tmap_wsf, tmap_asf, p, ctas, stream);
    case kTensor: return launch_mode<kTensor>(a_maps, tmap_w, tmap_wsf, tmap_asf, p, ctas, stream);
    case kMXFP8: return launch_mode<kMXFP8>(a_maps, tmap_w, tmap_wsf, tmap_asf, p, ctas, stream);
    case kMXFP4: return launch_mode<kMXFP4>(a_maps, tmap_w, tmap_wsf, tmap_asf, p, ctas, stream);
    case kMXFP8B32: return launch_mode<kMXFP8B32>(a_maps, tmap_w, tmap_wsf, tmap_asf, p, ctas, stream);
    case kMXFP4FP8A: return launch_mode<kMXFP4FP8A>(a_maps, tmap_w, tmap_wsf, tmap_asf, p, ctas, stream);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fg
