// Products grouped by expert in FP8_BLOCK128, many rows an expert: token tiles of up
// to 128 rows against 256 weight rows.  Schedule as in fg_grouped.cu.
//
// The fp32 scales (of a row of A and 128 K; of 128 weight rows and 128 K) cannot be
// the tensor core's, so every K step of 128 has a partial of its own, one of two
// in tensor memory, and eight warps fold each into registers, sum += a_s * b_s *
// partial, while the next is multiplied: the same operations in the same order as
// the 32-row form's, so a row's bits do not depend on the form (but where that
// cuts the line of K steps).  The tokens are the MMA's M side here, one row a
// lane, so that both scales are one factor a thread and K step: tokens on the N
// side would need a factor for every column, a multiply more for each value.  What
// that costs is a ragged tile's rest of 128 rows.
//
// What bounds it.  A step of 128 x 256 x 128 is 550 cycles of the tensor core, 48 KB
// from L2 to the SM (750 cycles) and the fold: each of four schedulers takes 256
// columns from tensor memory and folds them in 128 double multiply-adds, two warps
// at a time, whose waits do not cover one another's whole work: 900 cycles.  64
// experts, 4096 x 7168, 32768 rows in place: 805 us with as many for each expert
// (2.39 PFLOP/s), 887 unevenly; 4096 rows 295 us, the weights' bytes at 6.4 TB/s.
// Asking for the next step's first columns before this step's last are folded took
// 826 us to 805.  On pairs of SMs (256 x 256, 32 KB an SM and step) the fold holds
// it as it does here: 817 and 1006 us, and 423 for 346 at 128 rows an expert.  There
// a step without the fold's arithmetic would take 671 of 832 us, without its reads
// 652, without both 586.  Sixteen warps of 64 columns each, with the factors from two
// warps of their own, took 840 for 805: it is the work that adds up, not its latency.
//
// Gathered rows are laid out one after the other by a kernel before this one (55 us
// for 32768 rows of 7168).  Copied by the idle warps here they held the product up:
// four by their index to a tensor copy, 1251 us instead of 800; 16 bytes at a time
// by 64 threads, 1310.
//
// Registers: a thread keeps 128 sums and two times 32 values on their way from
// tensor memory, more than an even split of the file gives: the first warpgroup
// (copies, MMAs, two idle warps) gives its registers up.  The compiler, which counts
// with the 168 of the launch, reports 60 bytes a thread as spilled (72 loaded); where,
// it does not say.
#include <cuda_bf16.h>

#include "fg_grouped.cuh"
#include "fg_ptx.cuh"
#include "fg_tiles.cuh"

namespace fg {

namespace {

constexpr int TT = 128;
constexpr int kBlockThreads = 384;
constexpr int kRegsLow = 40, kRegsHigh = 232;
static_assert(128 * kRegsLow + 256 * kRegsHigh <= kBlockThreads * 168, "register split over the launch");
constexpr int kStages = 4;
constexpr int kTokBytes = TT * 128;
constexpr int kStageBytes = kTokBytes + 2 * kSlabBytes;
constexpr int kCols = 256;                 // weight rows of a unit, columns of a partial
constexpr int kTmemCols = 2 * kCols;
constexpr int kOutBytes = 32 * 64;         // per result warp: 32 rows x 32 columns of Y
constexpr int smem_bytes(int E) { return kStages * kStageBytes + 8 * kOutBytes + 1024 + 8 * (E + 1); }
static_assert(smem_bytes(kMaxExperts) <= 232448 - 1024, "shared memory budget");

__device__ __forceinline__ uint64_t splat2(float w) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(w));
  return r;
}

// a0 += v0 * w, a1 += v1 * w, each rounded once.  Volatile, so that they stay between
// the load of the next values and the wait for it.
__device__ __forceinline__ void fma2(float& a0, float& a1, uint32_t v0, uint32_t v1, uint64_t w2) {
  asm volatile("{\n .reg .b64 a, v;\n mov.b64 a, {%0, %1};\n mov.b64 v, {%2, %3};\n"
      " fma.rn.f32x2 a, v, %4, a;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(a0), "+f"(a1)
      : "r"(v0), "r"(v1), "l"(w2));
}

// a_maps: A's rows, or the gathered ones laid out; p.rows: whose scales they have.
__global__ void __launch_bounds__(kBlockThreads, 1)
    grouped_block_kernel(const __grid_constant__ AMaps a_maps, const GroupedParams p) {
  extern __shared__ uint8_t dsmem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[kStages], empty_bar[kStages];
  __shared__ __align__(8) uint64_t pfull_bar[2], pempty_bar[2];  // the two partials
  __shared__ __align__(8) uint64_t stall_bar, drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, issued_sh, consumed_sh;
  int* offs_sh = reinterpret_cast<int*>(smem + kStages * kStageBytes + 8 * kOutBytes);
  int* tiles_sh = offs_sh + p.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t T = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&full_bar[i], 1);
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&pfull_bar[i], 1);
      mbar_init(&pempty_bar[i], 8);  // the eight result warps
    }
    mbar_init(&stall_bar, 1);
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    issued_sh = 0;
    consumed_sh = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, kTmemCols);
    tmem_relinquish();
  }
  if (warp == 0 && lane < 8) prefetch_tmap(&a_maps.rows[lane]);
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  read_offsets<TT>(p.offsets, p.R, p.E, offs_sh, tiles_sh);
  tc_fence_before();
  __syncthreads();
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
  auto unit = [&](long long u) { return uniform(unit_at<TT>(s, u)); };
  auto slabs_of = [&](const Unit& q) { return min(2, wtiles - 2 * q.nt); };  // weight tiles of a unit

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
      // -------------------------------------------------------------- copies
      int it = 0;
      bool ok = true;
      for (long long u = blockIdx.x; ok && u < s.units; u += gridDim.x) {
        const Unit q = unit(u);
        const int n = slabs_of(q);
        const size_t slab = (static_cast<size_t>(q.e) * wtiles + 2 * q.nt) * s.KB;
        const CUtensorMap* a_map = &a_maps.rows[q.width / 16 - 1];
        const uint32_t bytes = q.width * 128 + n * kSlabBytes;
        for (int kb = 0; kb < s.KB; ++kb, ++it) {
          const int slot = it % kStages;
          ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[slot], ((it / kStages) & 1) ^ 1u, T, p.err, 91));
          if (!ok) break;
          uint8_t* st = smem + slot * kStageBytes;
          if (elect_one()) {
            mbar_arrive_expect_tx(&full_bar[slot], bytes);
            tma_load_2d(st, a_map, kb * 128, q.row0, &full_bar[slot]);
            for (int h = 0; h < n; ++h)
              bulk_g2s(st + kTokBytes + h * kSlabBytes, p.b_img + (slab + static_cast<size_t>(h) * s.KB + kb) * kSlabBytes, kSlabBytes,
                       &full_bar[slot]);
          }
          __syncwarp();
        }
      }
      if (lane == 0) {
        issued_sh = it;
        if (!ok) abort_sh = 1;
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMAs
      bool ok = true;
      if (p.debug_stall) ok = __all_sync(0xffffffffu, mbar_wait(&stall_bar, 0, T, p.err, 92));
      int it = 0;
      for (long long u = blockIdx.x; ok && u < s.units; u += gridDim.x) {
        const uint32_t idesc = idesc_e4m3(TT, 128 * slabs_of(unit(u)));
        for (int kb = 0; kb < s.KB; ++kb) {
          const int slot = it % kStages, b = it & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[slot], (it / kStages) & 1, T, p.err, 93));
          if (!ok) break;
          ok = __all_sync(0xffffffffu, mbar_wait(&pempty_bar[b], ((it >> 1) & 1) ^ 1u, T, p.err, 94));
          ++it;  // this stage's copies have landed
          if (!ok) break;
          tc_fence_after();
          const uint32_t st = smem_u32(smem) + slot * kStageBytes;
          if (elect_one()) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_f8f6f4(tmem + b * kCols, sdesc_sw128(st + j * 32), sdesc_sw128(st + kTokBytes + j * 32), idesc, j > 0 ? 1u : 0u);
            tc_commit(&pfull_bar[b]);     // the step's partial is ready
            tc_commit(&empty_bar[slot]);  // and its stage may be filled again
          }
          __syncwarp();
        }
      }
      if (lane == 0) {
        consumed_sh = it;
        if (!ok) abort_sh = 1;
      }
      if (it > 0) {  // every MMA and commit has landed before the block lets go of its memory
        if (elect_one()) tc_commit(&drain_bar);
        __syncwarp();
        mbar_wait(&drain_bar, 0, T, p.err, 95);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    // ---------------------------------------------------------------- results
    // lanes 32 qd .. + 31 of the tile, and one of the unit's two weight tiles
    const int qd = warp & 3, half = (warp - 4) >> 2;
    const int KS = p.K / 128;
    const float* a_s = static_cast<const float*>(p.a_scales);
    // scales are read four steps at a time, a group ahead of their use
    const bool vec4 = KS % 4 == 0 && ((reinterpret_cast<uintptr_t>(a_s) | reinterpret_cast<uintptr_t>(p.b_s)) & 15) == 0;
    uint8_t* stg = smem + kStages * kStageBytes + (warp - 4) * kOutBytes;
    // scale rows of unit q for this thread (rows and tiles past the end take the last; nothing of them is stored)
    auto scale_rows = [&](const Unit& q, const float*& arow, const float*& bcol) {
      int row = q.row0 + min(qd * 32 + lane, q.count - 1);
      if (p.rows) row = min(max(__ldg(p.rows + row), 0), p.T - 1);
      arow = a_s + static_cast<size_t>(row) * KS;
      bcol = p.b_s + (static_cast<size_t>(q.e) * wtiles + min(2 * q.nt + half, wtiles - 1)) * KS;
    };
    auto load_group = [&](const float* arow, const float* bcol, int kb0, float4& an, float4& bn) {
      if (vec4) {
        an = __ldg(reinterpret_cast<const float4*>(arow + kb0));
        bn = __ldg(reinterpret_cast<const float4*>(bcol + kb0));
      } else {
        an.x = __ldg(arow + kb0);
        bn.x = __ldg(bcol + kb0);
        an.y = kb0 + 1 < KS ? __ldg(arow + kb0 + 1) : 0.f;
        bn.y = kb0 + 1 < KS ? __ldg(bcol + kb0 + 1) : 0.f;
        an.z = kb0 + 2 < KS ? __ldg(arow + kb0 + 2) : 0.f;
        bn.z = kb0 + 2 < KS ? __ldg(bcol + kb0 + 2) : 0.f;
        an.w = kb0 + 3 < KS ? __ldg(arow + kb0 + 3) : 0.f;
        bn.w = kb0 + 3 < KS ? __ldg(bcol + kb0 + 3) : 0.f;
      }
    };
    const float* arow = a_s;
    const float* bcol = p.b_s;
    float4 an = make_float4(0.f, 0.f, 0.f, 0.f), bn = an;
    Unit q = {};
    if (blockIdx.x < s.units) {
      q = unit(blockIdx.x);
      scale_rows(q, arow, bcol);
      load_group(arow, bcol, 0, an, bn);
    }
    int it = 0;
    bool ok = true;
    uint32_t v[2][32];
    // wait for partial `it` and ask for its first columns
    auto begin = [&] {
      ok = __all_sync(0xffffffffu, mbar_wait(&pfull_bar[it & 1], (it >> 1) & 1, T, p.err, 96));
      tc_fence_after();
      if (ok) tmem_ld32(tmem + (it & 1) * kCols + half * 128 + (static_cast<uint32_t>(qd * 32) << 16), v[0]);
    };
    for (long long u = blockIdx.x; ok && u < s.units; u += gridDim.x) {
      const float* ar = arow;
      const float* bc = bcol;
      Unit next = q;
      float acc[128];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i] = 0.f;
      begin();
#pragma unroll 1
      for (int kb0 = 0; ok && kb0 < s.KB; kb0 += 4) {
        const float wg[4] = {an.x * bn.x, an.y * bn.y, an.z * bn.z, an.w * bn.w};
        // the next group's scales (the next unit's first) load while this group runs
        if (kb0 + 4 < s.KB) {
          load_group(ar, bc, kb0 + 4, an, bn);
        } else if (u + gridDim.x < s.units) {
          next = unit(u + gridDim.x);
          scale_rows(next, arow, bcol);
          load_group(arow, bcol, 0, an, bn);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (kb0 + j >= s.KB || !ok) break;
          const int b = it & 1;
          const uint32_t taddr = tmem + b * kCols + half * 128 + (static_cast<uint32_t>(qd * 32) << 16);
          const uint64_t w2 = splat2(wg[j]);
          // four 32-column loads, each folded while the next, or the next step's
          // first, is on its way
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            tmem_wait_ld();
            if (c < 3) {
              tmem_ld32(taddr + 32 * (c + 1), v[(c + 1) & 1]);
            } else {
              // the whole partial is in registers: the buffer may take the step after next
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&pempty_bar[b]);
              ++it;
              if (kb0 + j + 1 < s.KB) begin();
            }
#pragma unroll
            for (int i = 0; i < 32; i += 2) fma2(acc[32 * c + i], acc[32 * c + i + 1], v[c & 1][i], v[c & 1][i + 1], w2);
          }
        }
      }
      if (!ok) break;
      if (2 * q.nt + half < wtiles) {
        // bf16 rows through shared memory, 32 columns at a time (16-byte piece i of
        // row j at i ^ (j / 2 % 4)), out in 16-byte stores of the tile's own rows
        __nv_bfloat16* out = p.y + static_cast<size_t>(q.row0 + qd * 32) * p.N + (2 * q.nt + half) * 128;
        const int rows = q.count - qd * 32;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (rows <= 0) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 o;
            o.x = pack_bf16x2(acc[32 * r + 8 * j + 0], acc[32 * r + 8 * j + 1]);
            o.y = pack_bf16x2(acc[32 * r + 8 * j + 2], acc[32 * r + 8 * j + 3]);
            o.z = pack_bf16x2(acc[32 * r + 8 * j + 4], acc[32 * r + 8 * j + 5]);
            o.w = pack_bf16x2(acc[32 * r + 8 * j + 6], acc[32 * r + 8 * j + 7]);
            *reinterpret_cast<uint4*>(stg + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = o;
          }
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int row = 8 * j + (lane >> 2), piece = lane & 3;
            const uint4 o = *reinterpret_cast<const uint4*>(stg + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4));
            if (row < rows) *reinterpret_cast<uint4*>(out + static_cast<size_t>(row) * p.N + 32 * r + 8 * piece) = o;
          }
          __syncwarp();
        }
      }
      q = next;
    }
    if (!ok && lane == 0) abort_sh = 1;
  }

  // --------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (abort_sh && threadIdx.x == 0) {
    for (int it = consumed_sh; it < issued_sh; ++it)
      mbar_wait(&full_bar[it % kStages], (it / kStages) & 1, T, nullptr, 0);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace

cudaError_t launch_grouped_block(const AMaps& a_maps, const GroupedParams& p, int ctas, cudaStream_t stream) {
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(&grouped_block_kernel), smem_bytes(kMaxExperts));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kBlockThreads);
  cfg.dynamicSmemBytes = smem_bytes(p.E);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, grouped_block_kernel, a_maps, p);
}

}  // namespace fg
