// Products grouped by expert: Y[i] = A[rows[i]] . B_e^T for the rows i of
// expert e, offsets[e] <= i < offsets[e+1], with ragged counts known only on
// the device.
//
// Orientation.  The weight is the MMA's M operand (128 of its rows per tile,
// one 128 x 128-byte slab of the preshuffled image per K step) and the tokens
// its N operand, so a ragged expert costs what it holds: the instruction's N
// is set per tile to the tile's rows, rounded up to 16.  The accumulator (128
// lanes x up to TT fp32 columns) lives in tensor memory.
//
// Schedule.  Every block reads the offsets and sums, per expert, its token
// tiles (an expert's rows are cut into as few tiles of at most TT rows as hold
// them, of equal size); a unit is one token tile x one weight tile.  Units run
// expert by expert, the token tiles of one weight tile next to one another, so
// the blocks that share a weight tile take it at the same time and HBM moves
// it once.  No work is launched for experts without rows, and nothing comes
// back to the host.
//
//  - Many rows an expert (TT = 256): units of two weight tiles are dealt out
//    whole to pairs of SMs (fg_grouped_pair.cu).  Bound by the tensor cores and
//    the weights' bytes from HBM.  A first kernel lays out what every weight tile
//    reads again: the gathered rows one after the other (tensor copies of four
//    indexed rows each took three times as long as the product itself: 1797 us
//    against 624 us for 32768 mxfp4 rows, 4096 x 7168), and the token scales as
//    the atoms the tensor core reads.  FP8_BLOCK128: units of 128 rows and two
//    weight tiles on one SM (TT = 128, fg_grouped_block.cu).
//  - Few (TT = 32, decoding; this file): bound by the weights' bytes from HBM,
//    whatever the rows.  Where dealing whole units to the blocks would leave
//    much idle, the K steps of all units form one line that is cut evenly over
//    the blocks, wherever the cuts fall, so that all SMs stream to the end.
//    Blocks that share a unit leave fp32 partials in the workspace; the last to
//    arrive adds them in the order of K (the same bits each time) and stores.
//    Nobody waits for another block.  Measured, 4096 x 7168 of 64 experts, one
//    token x 8: mxfp8 40 us, fp8 x fp4 27, mxfp4 25, where the bytes alone take 35,
//    18 and 18: 4 us before the first K step (offsets, row indexes, the first
//    bytes) and 4 between one call's last store and the next one's start.  61
//    tokens, 7168 x 2048: 138 us, 6.5 TB/s by the bytes that HBM moves.
//
// Warp roles: 0 copies (weights by bulk copy, tokens by tensor copy: boxes of
// 16 rows, or four rows at a time by their index where rows are gathered);
// 1 issues the MMAs; 2-3 build the token scale atoms of the MX modes from the
// caller's E8M0 bytes; the others take the results out.
#include <cuda_bf16.h>

#include <algorithm>
#include <cstring>

#include "fg_grouped.cuh"
#include "fg_host.cuh"
#include "fg_internal.cuh"
#include "fg_ptx.cuh"

namespace fg {

namespace {

constexpr int kMinSlabs = 4;    // K steps a block of the cut line takes at least
constexpr int kShareSteps = 12;  // see the schedule
constexpr unsigned long long kGaveUp = 0x8000;  // of a ticket: a block of the unit gave up

constexpr int TT = 32;           // rows of a token tile
constexpr int kThreads = 256;    // copies, MMAs, two warps of scales, four of results
constexpr int kBlocksPerSm = 2;

constexpr bool smem_fits(int bytes) { return kBlocksPerSm * (bytes + 1024 + 256) <= 233472; }

template <int MODE>
struct GCfg {
  static constexpr int APS = MODE == kMXFP4 ? 2 : (is_mx(MODE) ? 1 : 0);
  // fp8 x fp4 moves half a stage's bytes from HBM: one stage more (28.5 -> 28.2 us
  // for one token, 103 -> 100 us for eight); the 8-bit modes lost 2-4 % with it
  static constexpr int STAGES = MODE == kMXFP4FP8A ? 5 : 4;
  static constexpr int TOK_BYTES = TT * 128;
  static constexpr int SFW_BYTES = APS * 512;
  static constexpr int SFT_BYTES = APS * 512;
  static constexpr int STAGE_RAW = kSlabBytes + TOK_BYTES + SFW_BYTES + SFT_BYTES;
  static constexpr int STAGE_BYTES = (STAGE_RAW + 1023) / 1024 * 1024;
  static constexpr int SF_COLS = APS * 4;  // of each operand
  // FP8_BLOCK128's fp32 scales cannot be the MMA's: every K step (one scale
  // block) has an accumulator of its own, four in turn, which the result warps
  // fold into registers with its scales
  static constexpr bool FOLD = MODE == kBlock;
  static constexpr int ACCS = FOLD ? 4 : 2;
  static constexpr int ACC_COLS = ACCS * TT;
  static constexpr int TMEM_NEED = ACC_COLS + STAGES * 2 * SF_COLS;
  static constexpr int TMEM_COLS = TMEM_NEED <= 64 ? 64 : (TMEM_NEED <= 128 ? 128 : 256);
  // with the schedule of E experts: two blocks an SM up to 500 experts
  static constexpr int smem(int E) { return STAGES * STAGE_BYTES + 1024 + 8 * (E + 1); }
  static_assert(TMEM_NEED <= TMEM_COLS && kBlocksPerSm * TMEM_COLS <= 512, "TMEM budget");
  static_assert(smem_fits(STAGES * STAGE_BYTES + 1024 + 8 * 501), "shared memory budget");
};

// One block's share of a unit: K steps [k0, k1).
struct Share {
  long long u;
  int k0, k1;
};

// Cut c of the line of W steps over `blocks` blocks, and the block that holds step x.
__device__ __forceinline__ long long cut_at(const Schedule& s, int c) { return s.W * c / s.blocks; }
__device__ __forceinline__ int holder_of(const Schedule& s, long long x) {
  return static_cast<int>(((x + 1) * s.blocks + s.W - 1) / s.W) - 1;
}

__device__ __forceinline__ int share_count(const Schedule& s) {
  if (!s.cut) return s.c < s.units ? static_cast<int>((s.units - s.c + s.blocks - 1) / s.blocks) : 0;
  return s.hi > s.lo ? static_cast<int>((s.hi - 1) / s.KB - s.lo / s.KB + 1) : 0;
}

__device__ __forceinline__ Share share_at(const Schedule& s, int i) {
  Share h;
  if (!s.cut) {
    h.u = s.c + static_cast<long long>(i) * s.blocks;
    h.k0 = 0;
    h.k1 = s.KB;
    return h;
  }
  h.u = s.lo / s.KB + i;
  const long long first = h.u * s.KB;
  h.k0 = i == 0 ? static_cast<int>(s.lo - first) : 0;
  h.k1 = static_cast<int>(min(static_cast<long long>(s.KB), s.hi - first));
  return h;
}

template <int MODE>
__device__ __forceinline__ void mma_step(uint32_t d, uint64_t a, uint64_t b, int n, int j, int kb, uint32_t sfw,
                                         uint32_t sft, uint32_t accum) {
  if (MODE == kBF16) {
    mma_f16(d, a, b, idesc_bf16(128, n), accum);
  } else if (MODE == kTensor || MODE == kBlock) {
    mma_f8f6f4(d, a, b, idesc_e4m3(128, n), accum);
  } else if (MODE == kMXFP8) {
    // the weight's byte of its four-slab atom; the token atoms have the slab's
    // scale in all four
    mma_mxf8f6f4(d, a, b, idesc_mx(128, n, kF8f6f4E4M3, kb & 3, j), sfw, sft, accum);
  } else if (MODE == kMXFP8B32) {
    mma_mxf8f6f4(d, a, b, idesc_mx(128, n, kF8f6f4E4M3, j, j), sfw, sft, accum);
  } else if (MODE == kMXFP4FP8A) {
    mma_mxf8f6f4(d, a, b, idesc_mx_ab(128, n, kF8f6f4E2M1, kF8f6f4E4M3, j, j), sfw, sft, accum);
  } else {
    const int g = j >> 1, id = 2 * (j & 1);
    mma_mxf4(d, a, b, idesc_mx(128, n, kMxf4E2M1, id, id), sfw + 4 * g, sft + 4 * g, accum);
  }
}

// tmap_b: fp8 x fp4 only, the weight image's blocks.
template <int MODE, bool GATHER>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm)
    grouped_kernel(const __grid_constant__ AMaps a_maps, const __grid_constant__ CUtensorMap tmap_b,
                   const GroupedParams p) {
  using C = GCfg<MODE>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t dsmem[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~uintptr_t(1023));
  __shared__ __align__(8) uint64_t full_bar[ST], empty_bar[ST];
  __shared__ __align__(8) uint64_t accf_bar[C::ACCS], acce_bar[C::ACCS];
  __shared__ __align__(8) uint64_t stall_bar, drain_bar;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, issued_sh, consumed_sh, last_sh;
  int* offs_sh = reinterpret_cast<int*>(smem + ST * C::STAGE_BYTES);
  int* tiles_sh = offs_sh + p.E + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint64_t T = p.timeout_ns;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&full_bar[i], C::APS ? 3 : 1);  // + one arrival per scale warp
      mbar_init(&empty_bar[i], 1);
    }
    for (int i = 0; i < C::ACCS; ++i) {
      mbar_init(&accf_bar[i], 1);
      mbar_init(&acce_bar[i], 4);
    }
    mbar_init(&stall_bar, 1);
    mbar_init(&drain_bar, 1);
    abort_sh = 0;
    issued_sh = 0;
    consumed_sh = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(&tmem_base_sh, C::TMEM_COLS);
    tmem_relinquish();
  }
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  if (warp == 0) {
    prefetch_tmap(&a_maps.rows[0]);
    if (MODE == kMXFP4FP8A) prefetch_tmap(&tmap_b);
  }
  read_offsets<TT>(p.offsets, p.R, p.E, offs_sh, tiles_sh);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;

  Schedule s;
  s.offs = offs_sh;
  s.tiles = tiles_sh;
  s.E = p.E;
  s.NT = p.N / 128;
  s.KB = p.KB;
  s.units = static_cast<long long>(tiles_sh[p.E]) * s.NT;
  s.W = s.units * s.KB;
  s.c = blockIdx.x;
  s.blocks = gridDim.x;
  // Whole units or a cut line?  Full rounds of whole units keep the memory
  // busy.  The units that remain take s.KB steps of a lone block's pace, which
  // kBusy blocks need to fill the memory; shared evenly they would take rem /
  // kBusy of that, plus the round of partials at the end, as long as kShareSteps
  // steps.  256 units on 304 blocks, K = 7168: 26.9 us whole, 30.6 cut (fp8 x fp4),
  // 40.3 and 45.6 (mxfp8); 105 units, 32 steps, mxfp8: 16 and 20; 112 units, 20 steps,
  // mxfp4: 12 and 18; 112 units of 25 rows, 56 steps, mxfp8: 27 and 22.
  {
    constexpr int kBusy = MODE == kMXFP4FP8A ? 216 : 137;
    const int rem = static_cast<int>(s.units % gridDim.x);
    s.cut = rem > 0 && rem < kBusy && static_cast<long long>(s.KB) * (kBusy - rem) > kShareSteps * kBusy;
  }
  if (s.cut) {
    const long long most = (s.W + kMinSlabs - 1) / kMinSlabs;
    s.blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), max(most, 1ll)));
    s.lo = s.c < s.blocks ? cut_at(s, s.c) : 0;
    s.hi = s.c < s.blocks ? cut_at(s, s.c + 1) : 0;
  }
  const int shares = share_count(s);

  if (warp == 0) {
    // ---------------------------------------------------------------- copies
    int it = 0;
    bool ok = true;
    for (int i = 0; ok && i < shares; ++i) {
      const Share h = share_at(s, i);
      const Unit q = uniform(unit_at<TT>(s, h.u));
      const long long wt = static_cast<long long>(q.e) * s.NT + q.nt;  // weight tile of the stacked image
      // rows that are copied; the accumulator's columns past them hold what
      // the rows of an earlier step left and are not stored
      const int copied = GATHER ? (q.count + 3) & ~3 : q.width;
      const uint32_t bytes = (MODE == kMXFP4FP8A ? kSlabBytes / 2 : kSlabBytes) + copied * 128 + C::SFW_BYTES;
      // the weight's part of a stage (one lane)
      auto weights = [&](int kb, int slot) {
        uint8_t* st = smem + slot * C::STAGE_BYTES;
        mbar_arrive_expect_tx(&full_bar[slot], bytes);
        const long long slab = wt * s.KB + kb;
        if (MODE == kMXFP4FP8A)
          tma_load_3d(st, &tmap_b, 0, 0, static_cast<int32_t>(slab), &full_bar[slot]);
        else
          bulk_g2s(st, p.b_img + slab * kSlabBytes, kSlabBytes, &full_bar[slot]);
        if (C::APS) {
          const long long atom = MODE == kMXFP8 ? wt * ((s.KB + 3) / 4) + kb / 4 : slab * C::APS;
          bulk_g2s(st + kSlabBytes + C::TOK_BYTES, p.b_sf + atom * 512, C::SFW_BYTES, &full_bar[slot]);
        }
      };
      // gathered: the row of A for this lane's row of the tile; rows past the
      // tile's end repeat its last one, indexes are clamped into A
      int idx = 0;
      if (GATHER) idx = __ldg(p.rows + q.row0 + min(lane, q.count - 1));
      // the first stages are empty: their weights go out while the row indexes come
      const int early = GATHER && i == 0 ? min(ST, h.k1 - h.k0) : 0;
      if (early > 0) {
        if (elect_one()) {
          for (int j = 0; j < early; ++j) weights(h.k0 + j, j);
        }
        __syncwarp();
      }
      // ... all of them in every lane, four to a copy
      int rows4[TT / 4][4];
      if (GATHER) {
        idx = min(max(idx, 0), p.T - 1);
#pragma unroll
        for (int g = 0; g < TT / 4; ++g)
#pragma unroll
          for (int j = 0; j < 4; ++j) rows4[g][j] = __shfl_sync(0xffffffffu, idx, 4 * g + j);
      }
      for (int kb = h.k0; kb < h.k1; ++kb, ++it) {
        const int slot = it % ST;
        ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[slot], ((it / ST) & 1) ^ 1u, T, p.err, 61));
        if (!ok) break;
        uint8_t* st = smem + slot * C::STAGE_BYTES;
        uint8_t* tok = st + kSlabBytes;
        if (elect_one()) {
          if (it >= early) weights(kb, slot);
          if (GATHER) {
#pragma unroll
            for (int g = 0; g < TT / 4; ++g)
              if (4 * g < copied) tma_gather4(tok + g * 512, &a_maps.rows[0], kb * 128, rows4[g], &full_bar[slot]);
          } else {
            tma_load_2d(tok, &a_maps.rows[q.width > 16 ? 1 : 0], kb * 128, q.row0, &full_bar[slot]);
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
    // ------------------------------------------------------------------ MMAs
    bool ok = true;
    if (p.debug_stall) ok = __all_sync(0xffffffffu, mbar_wait(&stall_bar, 0, T, p.err, 62));
    int it = 0;
    for (int i = 0; ok && i < shares; ++i) {
      const Share h = share_at(s, i);
      const Unit q = uniform(unit_at<TT>(s, h.u));
      // accumulators are taken in turn by share, or by K step (FOLD)
      const int acc = i & 1;
      uint32_t d = tmem + acc * TT;
      if (!C::FOLD) {
        ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar[acc], ((i >> 1) & 1) ^ 1u, T, p.err, 63));
        if (!ok) break;
        tc_fence_after();
      }
      for (int kb = h.k0; kb < h.k1; ++kb, ++it) {
        const int slot = it % ST;
        ok = __all_sync(0xffffffffu, mbar_wait(&full_bar[slot], (it / ST) & 1, T, p.err, 64));
        if (!ok) break;
        const int part = it % C::ACCS;
        if (C::FOLD) {
          ok = __all_sync(0xffffffffu, mbar_wait(&acce_bar[part], ((it / C::ACCS) & 1) ^ 1u, T, p.err, 63));
          if (!ok) {
            ++it;  // this step's copies have landed
            break;
          }
          d = tmem + part * TT;
        }
        tc_fence_after();
        const uint32_t st = smem_u32(smem) + slot * C::STAGE_BYTES;
        const uint32_t sfw = tmem + C::ACC_COLS + slot * 2 * C::SF_COLS;
        const uint32_t sft = sfw + C::SF_COLS;
        if (elect_one()) {
          if (C::APS) {
            const uint32_t sw = st + kSlabBytes + C::TOK_BYTES;
            const uint32_t stk = sw + C::SFW_BYTES;
#pragma unroll
            for (int g = 0; g < C::APS; ++g) {
              tc_cp_32x128b_warpx4(sfw + 4 * g, sdesc_plain_rows16(sw + 512 * g));
              tc_cp_32x128b_warpx4(sft + 4 * g, sdesc_plain_rows16(stk + 512 * g));
            }
          }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_step<MODE>(d, sdesc_sw128(st + j * 32), sdesc_sw128(st + kSlabBytes + j * 32), q.width, j, kb, sfw, sft,
                           ((!C::FOLD && kb > h.k0) || j > 0) ? 1u : 0u);
          tc_commit(&empty_bar[slot]);
          if (C::FOLD) tc_commit(&accf_bar[part]);
        }
        __syncwarp();
      }
      if (!ok) break;
      if (!C::FOLD) {
        if (elect_one()) tc_commit(&accf_bar[acc]);
        __syncwarp();
      }
    }
    if (lane == 0) {
      // a step whose wait gave up was not consumed; the teardown waits for it
      consumed_sh = it;
      if (!ok) abort_sh = 1;
    }
    if (it > 0) {  // every MMA and commit has landed before the block lets go of its memory
      if (elect_one()) tc_commit(&drain_bar);
      __syncwarp();
      mbar_wait(&drain_bar, 0, T, p.err, 65);
    }
  } else if (warp < 4) {
    // ----------------------------------------------------- token scale atoms
    if (C::APS) {
      // thread (warp - 2, lane): row lane of the tile; the two warps share the
      // slab's atoms (mxfp4) or one of them only arrives
      const int g = warp - 2;
      const bool mine = g < C::APS;
      const uint8_t* asf = static_cast<const uint8_t*>(p.a_scales);
      const int cols = MODE == kMXFP8 ? p.K / 128 : p.K / 32;
      const bool words = (reinterpret_cast<uintptr_t>(asf) & 3u) == 0;
      int it = 0;
      bool ok = true;
      for (int i = 0; ok && i < shares; ++i) {
        const Share h = share_at(s, i);
        const Unit q = uniform(unit_at<TT>(s, h.u));
        int row = q.row0 + min(lane, q.count - 1);
        if (GATHER && mine) row = min(max(__ldg(p.rows + row), 0), p.T - 1);
        const uint8_t* src = asf + static_cast<size_t>(row) * cols;
        // the four E8M0 bytes of this warp's atom at K step kb
        auto word = [&](int kb) -> uint32_t {
          if (!mine) return 0u;
          if (MODE == kMXFP8) return static_cast<uint32_t>(__ldg(src + kb)) * 0x01010101u;
          const uint8_t* b = src + (kb * C::APS + g) * 4;
          if (words) return __ldg(reinterpret_cast<const uint32_t*>(b));
          return b[0] | (static_cast<uint32_t>(b[1]) << 8) | (static_cast<uint32_t>(b[2]) << 16) |
                 (static_cast<uint32_t>(b[3]) << 24);
        };
        uint32_t next = word(h.k0);
        for (int kb = h.k0; kb < h.k1; ++kb, ++it) {
          const int slot = it % ST;
          ok = __all_sync(0xffffffffu, mbar_wait(&empty_bar[slot], ((it / ST) & 1) ^ 1u, T, p.err, 66));
          if (!ok) break;
          uint8_t* sft = smem + slot * C::STAGE_BYTES + kSlabBytes + C::TOK_BYTES + C::SFW_BYTES;
          if (mine) *reinterpret_cast<uint32_t*>(sft + g * 512 + lane * 16) = next;
          if (kb + 1 < h.k1) next = word(kb + 1);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&full_bar[slot]);
        }
      }
      if (!ok && lane == 0) abort_sh = 1;
    }
  } else {
    // -------------------------------------------------------------- results
    const int qd = warp & 3;
    const float scale = MODE == kTensor ? __ldg(static_cast<const float*>(p.a_scales)) * __ldg(p.b_s) : 1.f;
    bool ok = true;
    int it = 0;  // K steps so far (FOLD)
    // One thread's arrival at a shared unit, when the block's partial is in the
    // workspace; last_sh: this block adds up.  A ticket holds the call's tag, a
    // bit for a block that gave up, and the arrivals; a word of another call (or
    // of nothing) counts as none.  Every block arrives, also one that gave up,
    // and the last leaves the word clear: a replay of a captured call carries
    // the same tag and must not find the arrivals of an earlier run.  The
    // barrier before the call put the block's partial before this thread, its
    // fence puts it before the arrival.  First guess: the word is clear, as a
    // finished unit leaves it.
    auto arrive = [&](long long u, bool gave_up) {
      const long long first = u * s.KB;
      const int c0 = holder_of(s, first), others = holder_of(s, first + s.KB - 1) - c0;
      __threadfence();
      unsigned long long* t = p.tickets + c0;
      unsigned long long old = 0ull, seen, held;
      int arrived;
      bool last;
      do {
        seen = old;
        held = (seen >> 16) == p.epoch ? seen & 0xffffu : 0ull;
        arrived = static_cast<int>(held & (kGaveUp - 1));
        last = arrived == others;
        held = (held & kGaveUp) | (gave_up ? kGaveUp : 0ull);
        old = atomicCAS(t, seen, last ? 0ull : (p.epoch << 16) | held | static_cast<unsigned long long>(arrived + 1));
      } while (old != seen);
      __threadfence();
      last_sh = last && held == 0ull;
    };
    for (int i = 0; i < shares; ++i) {
      const Share h = share_at(s, i);
      const Unit q = uniform(unit_at<TT>(s, h.u));
      const int acc = i & 1;
      // a warp that gave up waits for nothing more, but still meets the others
      // at the barriers of the shared units
      const bool shared_unit = h.k0 > 0 || h.k1 < s.KB;  // of a cut line
      uint32_t v[TT];
      if (C::FOLD) {
        // lane m has the scales of row m of the tile, all lanes the weight
        // tile's; each is loaded a step ahead
        int row = q.row0 + min(lane, q.count - 1);
        if (GATHER) row = min(max(__ldg(p.rows + row), 0), p.T - 1);
        const float* as = static_cast<const float*>(p.a_scales) + static_cast<size_t>(row) * s.KB;
        const float* bs = p.b_s + (static_cast<size_t>(q.e) * s.NT + q.nt) * s.KB;
        float a_next = ld_nc_f32(as + h.k0), b_next = ld_nc_f32(bs + h.k0);
        float sum[TT];
#pragma unroll
        for (int m = 0; m < TT; ++m) sum[m] = 0.f;
        for (int kb = h.k0; ok && kb < h.k1; ++kb, ++it) {
          const float w = a_next * b_next;
          if (kb + 1 < h.k1) {
            a_next = ld_nc_f32(as + kb + 1);
            b_next = ld_nc_f32(bs + kb + 1);
          }
          const int part = it % C::ACCS;
          ok = __all_sync(0xffffffffu, mbar_wait(&accf_bar[part], (it / C::ACCS) & 1, T, p.err, 67));
          if (!ok) break;
          tc_fence_after();
          tmem_ld32(tmem + part * TT + (static_cast<uint32_t>(qd * 32) << 16), v);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acce_bar[part]);
#pragma unroll
          for (int m = 0; m < TT; ++m) sum[m] = fmaf(__shfl_sync(0xffffffffu, w, m), __uint_as_float(v[m]), sum[m]);
        }
#pragma unroll
        for (int m = 0; m < TT; ++m) v[m] = __float_as_uint(sum[m]);
      } else if (ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(&accf_bar[acc], (i >> 1) & 1, T, p.err, 67));
        if (ok) {
          tc_fence_after();
          tmem_ld32(tmem + acc * TT + (static_cast<uint32_t>(qd * 32) << 16), v);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&acce_bar[acc]);
        }
      }
      if (!ok) {
        if (lane == 0) abort_sh = 1;
        if (shared_unit) {
          bar_sync_named(1, 128);
          if (threadIdx.x == 128) arrive(h.u, true);
          bar_sync_named(1, 128);
        }
        continue;
      }
      const int n = qd * 32 + lane;  // row of the weight tile
      if (shared_unit) {
        // a shared unit: leave the partial, and let the last to arrive add up
        const long long first = h.u * s.KB;
        const int c0 = holder_of(s, first), c1 = holder_of(s, first + s.KB - 1);
        const size_t tile = static_cast<size_t>(TT) * 128;
        // a block's share that begins inside a unit is its first, slot 0; one
        // that begins with the unit and ends inside it is its last, slot 1
        float* mine = p.part + (2 * static_cast<size_t>(s.c) + (h.k0 > 0 ? 0 : 1)) * tile;
#pragma unroll
        for (int m = 0; m < TT; ++m)
          if (m < q.count) __stcg(mine + m * 128 + n, __uint_as_float(v[m]));
        bar_sync_named(1, 128);
        if (threadIdx.x == 128) arrive(h.u, *reinterpret_cast<volatile int*>(&abort_sh) != 0);
        bar_sync_named(1, 128);
        const bool last = last_sh != 0;
        if (!last) continue;
        // in the order of K; a partial's rows are all on their way before the
        // first is added
        const float* part = p.part + (2 * static_cast<size_t>(c0) + 1) * tile + n;
#pragma unroll
        for (int m = 0; m < TT; ++m)
          if (m < q.count) v[m] = __float_as_uint(__ldcg(part + m * 128));
#pragma unroll 1
        for (int c = c0 + 1; c <= c1; ++c) {
          part = p.part + 2 * static_cast<size_t>(c) * tile + n;
          float w[TT];
#pragma unroll
          for (int m = 0; m < TT; ++m) w[m] = m < q.count ? __ldcg(part + m * 128) : 0.f;
#pragma unroll
          for (int m = 0; m < TT; ++m) v[m] = __float_as_uint(__uint_as_float(v[m]) + w[m]);
        }
      }
      __nv_bfloat16* out = p.y + static_cast<size_t>(q.row0) * p.N + q.nt * 128 + n;
#pragma unroll
      for (int m = 0; m < TT; ++m)
        if (m < q.count) out[static_cast<size_t>(m) * p.N] = __float2bfloat16_rn(__uint_as_float(v[m]) * scale);
    }
  }

  // --------------------------------------------------------------- teardown
  tc_fence_before();
  __syncthreads();
  if (abort_sh && threadIdx.x == 0) {
    for (int it = consumed_sh; it < issued_sh; ++it)
      mbar_wait(&full_bar[it % ST], (it / ST) & 1, T, nullptr, 0);
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, C::TMEM_COLS);
}

// What TT = 128 and 256 lay out first: the gathered rows of A (a_rows) and the token
// scale atoms (a_sf), each where wanted.
struct PrepParams {
  const uint8_t* a;
  const uint8_t* scales;
  const int32_t* offsets;
  const int32_t* rows;
  uint8_t* a_rows;  // [R][rb] or null
  uint8_t* a_sf;    // [tile][NA][128-row block of the tile][512] (null: no MX scales)
  int T, R, E;
  int rb;           // bytes of a row of A
  int sb;           // scale bytes of a row
  int NA;           // atoms of a 128-row block: four scale bytes of each row to an atom
  int copy_blocks;  // the first blocks copy rows, the others build atoms
};

constexpr int kPrepRows = 4;  // rows a copying block has in flight, 64 threads each

__global__ void __launch_bounds__(256) grouped_prep_kernel(const PrepParams p) {
  extern __shared__ int sched_sh[];
  pdl_wait();
  pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) < p.copy_blocks) {
    // two rows at a time, so that both rows' loads are in flight together
    const int lane = threadIdx.x & 63, chunks = p.rb / 16;
    const int64_t step = static_cast<int64_t>(p.copy_blocks) * kPrepRows;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kPrepRows + (threadIdx.x >> 6); i < p.R; i += 2 * step) {
      const int64_t at[2] = {i, i + step};
      const uint4* src[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = at[r] < p.R ? min(max(__ldg(p.rows + at[r]), 0), p.T - 1) : 0;
        src[r] = reinterpret_cast<const uint4*>(p.a + static_cast<size_t>(row) * p.rb);
      }
      for (int c0 = lane; c0 < chunks; c0 += 4 * 64) {
        uint4 v[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (at[r] < p.R && c0 + j * 64 < chunks) v[r][j] = __ldg(src[r] + c0 + j * 64);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (at[r] < p.R && c0 + j * 64 < chunks)
              reinterpret_cast<uint4*>(p.a_rows + static_cast<size_t>(at[r]) * p.rb)[c0 + j * 64] = v[r][j];
      }
    }
    return;
  }
  constexpr int BLOCKS = 2;  // 128-row blocks of a tile
  int* offs = sched_sh;
  int* tiles = sched_sh + p.E + 1;
  read_offsets<256>(p.offsets, p.R, p.E, offs, tiles);
  Schedule s;
  s.offs = offs;
  s.tiles = tiles;
  s.E = p.E;
  s.NT = 1;
  // A thread takes four atoms in a row of one line: byte 16 * line + 4 * b + j
  // of an atom belongs to row 32 * b + line of its 128, scale byte 4 * atom + j.
  const int quads = (p.NA + 3) / 4;
  const bool whole = (p.sb & 15) == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15u) == 0;
  const int64_t total = static_cast<int64_t>(tiles[p.E]) * quads * (32 * BLOCKS);
  const int64_t step = static_cast<int64_t>(gridDim.x - p.copy_blocks) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x - p.copy_blocks) * blockDim.x + threadIdx.x; i < total; i += step) {
    const int line = static_cast<int>(i & 31), blk = static_cast<int>(i >> 5) % BLOCKS;
    const int64_t tq = (i >> 5) / BLOCKS;
    const int tile = static_cast<int>(tq / quads), quad = static_cast<int>(tq - static_cast<int64_t>(tile) * quads);
    const Unit q = unit_at<256>(s, tile);
    if (blk * 128 >= q.width) continue;
    uint32_t w[4][4];  // [block of 32 rows][atom]
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int m = min(blk * 128 + b * 32 + line, q.count - 1);
      int row = q.row0 + m;
      if (p.rows) row = min(max(__ldg(p.rows + row), 0), p.T - 1);
      const uint8_t* src = p.scales + static_cast<size_t>(row) * p.sb + quad * 16;
      if (whole) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(src));
        w[b][0] = u.x; w[b][1] = u.y; w[b][2] = u.z; w[b][3] = u.w;
      } else {
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          w[b][a] = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (quad * 16 + a * 4 + j < p.sb) w[b][a] |= static_cast<uint32_t>(__ldg(src + a * 4 + j)) << (8 * j);
        }
      }
    }
#pragma unroll
    for (int a = 0; a < 4; ++a) {
      const int atom = quad * 4 + a;
      if (atom < p.NA)
        *reinterpret_cast<uint4*>(p.a_sf + ((static_cast<size_t>(tile) * p.NA + atom) * BLOCKS + blk) * 512 + line * 16) =
            make_uint4(w[0][a], w[1][a], w[2][a], w[3][a]);
    }
  }
}

template <int MODE, bool GATHER>
cudaError_t launch_one(const AMaps& a_maps, const CUtensorMap& tmap_b, const GroupedParams& p, int blocks,
                       cudaStream_t stream) {
  using C = GCfg<MODE>;
  auto* kernel = &grouped_kernel<MODE, GATHER>;
  cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), C::smem(kMaxExperts));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::smem(p.E);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, a_maps, tmap_b, p);
}

template <int MODE>
cudaError_t launch_mode(const AMaps& a_maps, const CUtensorMap& tmap_b, const GroupedParams& p, int blocks,
                        cudaStream_t stream) {
  return p.rows ? launch_one<MODE, true>(a_maps, tmap_b, p, blocks, stream)
                : launch_one<MODE, false>(a_maps, tmap_b, p, blocks, stream);
}

cudaError_t launch_prep(PrepParams p, int64_t tiles, cudaStream_t stream) {
  // blocks in proportion to the work, at most eight an SM for each part
  const int64_t most = 8 * static_cast<int64_t>(sm_count());
  const int64_t rows = p.a_rows ? (p.R + kPrepRows - 1) / kPrepRows : 0;
  const int64_t lines = p.a_sf ? (tiles * ((p.NA + 3) / 4) * 64 + 255) / 256 : 0;
  p.copy_blocks = static_cast<int>(rows < most ? rows : most);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.copy_blocks + (lines < most ? lines : most)));
  cfg.blockDim = dim3(256);
  cfg.dynamicSmemBytes = 8 * (p.E + 1);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, grouped_prep_kernel, p);
}

// Token tile, blocks (two for each pair of SMs) and workspace of a call: partials
// and tickets (tt 32), or scale atoms and gathered rows (tt 128, 256), in this order.
struct GroupedPlan {
  int tt, blocks;
  int64_t tiles;  // no more token tiles than this, however the rows fall
  int atoms;      // scale atoms of a 128-row block
  uint64_t part_bytes, ticket_bytes, sf_bytes, rows_bytes;
  uint64_t total() const {
    const uint64_t line = part_bytes + ticket_bytes, laid = sf_bytes + rows_bytes;
    return std::max(line, laid);
  }
};

// have: bytes of workspace that the call is given.
GroupedPlan grouped_plan(int mode, int64_t R, int64_t E, int64_t N, int64_t K, bool gather, uint64_t have = UINT64_MAX) {
  GroupedPlan g;
  memset(&g, 0, sizeof g);
  if (R == 0) return g;
  const int64_t KB = row_bytes(mode, K) / 128;
  // Token tiles of 32 rows or pairs of SMs with tiles of 256.  By the rows of an
  // expert on average (64 experts, 4096 x 7168, mxfp8): at 16 rows 326 us with 32
  // (experts above 32 rows read their weights again) and 290 on pairs; at 8 the
  // two are equal, and below that pairs idle.  But pairs share no unit, so a
  // call with fewer units than pairs leaves SMs without work, and the layout
  // kernel before them takes 3 us: there, or where the K steps are few, 32-row
  // tiles are faster up to about rows x pairs of weight tiles = 8000 (8 experts of
  // 512 x 7168: 25 rows each 20 us against 26, 100 rows 22 against 30; bf16 38 rows
  // 26 against 43; 4 of 1024 x 7168 mxfp4, 250 rows: 18 against 22; 16 of 128 x 2048,
  // 375 rows: 9 against 18; 8 of 2176 x 2048, 34 rows: 13 against 15; 64 of 2304 x
  // 256, 9 rows, 2 steps: 11 against 19; 8 of 2048 x 7168, 15 rows: 29 and 29).
  const int64_t wpairs = (N / 128 + 1) / 2, active = E < R ? E : R;
  const bool few = R * wpairs < 8000 && (active * wpairs < grouped_pair_clusters() || KB <= 8);
  const bool block = mode == FG_FP8_BLOCK128;
  g.tt = R <= 8 * E || few ? 32 : 256;
  // FP8_BLOCK128: tiles of 128 rows on one SM above 32 rows an expert, where 32-row
  // tiles read the weights again (64 experts, 4096 x 7168: 32 rows each 279 us with
  // 32 and 287 with 128, 48 rows 346 and 291, 512 rows 2640 and 805), unless they lose
  // that by idle SMs, or by the layout of gathered rows where a weight is narrow: what
  // a call takes is estimated for either.  Both spend 0.5 us on a block's K step and 1 us
  // on a unit; 32-row tiles are cut evenly over two blocks an SM, 128-row units of two
  // weight tiles go whole, half a round idle behind the first; half of the experts' last
  // tiles are counted.  Below four K steps a block of the cut line joins parts of several
  // units, which is the slower wherever they fall (one step, 32 experts of 384, 45 rows
  // each: 11.0 us with 32 and 6.2 with 128).
  // In 800 calls with random routing (2 to 128 experts of 128 x 128 to 4096 x 7168, 32 to
  // 600 rows each) this takes 1.006 times the faster form's time, 128-row tiles from 48
  // units on 1.040, 32-row tiles alone 1.33; it is slower than 32-row tiles by more than
  // 5 % in 14 of them (84 from 48 units on), at worst for 16 experts of 2304 x 4096, 42
  // rows each gathered: 38 us with 32 and 48 with 128.  64 experts of 128 x 7168, 300
  // rows gathered: 73 and 101 (32 chosen); 8 of 2048 x 4096, 97 rows: 33 and 20 (128).
  if (block) {
    const double sms = sm_count(), halves = 0.5 * static_cast<double>(active), unit = 0.5 * KB + 1.0;
    const double line = (R / 32.0 + halves) * static_cast<double>(N / 128) / (kBlocksPerSm * sms);
    const double whole = (R / 128.0 + halves) * static_cast<double>(wpairs) / sms;
    const double us32 = 5.7 + unit * line;
    const double us128 = 5.0 + unit * (whole > 1.0 ? whole + 0.5 : 1.0) + (gather ? 1.5 + 0.24e-6 * R * K : 0.0);
    g.tt = R > 32 * E && (KB < kMinSlabs || us128 < 0.96 * us32) ? 128 : 32;
    // (32-row tiles gather as they copy: a workspace without room for the rows will do)
    if (g.tt == 128 && gather && have < static_cast<uint64_t>(R * K)) g.tt = 32;
  }
  g.tiles = R / g.tt + active;
  const int64_t units = g.tiles * (g.tt == 32 ? N / 128 : wpairs);
  const int64_t line = ((R / 32 + active) * (N / 128) * KB + kMinSlabs - 1) / kMinSlabs;  // blocks of a line of 32-row tiles
  const int64_t most = kBlocksPerSm * static_cast<int64_t>(sm_count());
  g.blocks = static_cast<int>(g.tt == 32    ? std::min(line, most)
                              : g.tt == 128 ? std::min<int64_t>(units, sm_count())
                                            : 2 * std::min<int64_t>(units, grouped_pair_clusters()));
  if (g.tt == 32 || block) {
    // (FP8_BLOCK128's workspace is never less than with 32-row tiles alone: in
    // 128-row tiles the gathered rows begin where its partials would)
    g.part_bytes = static_cast<uint64_t>(std::min(line, most)) * 2 * 32 * 128 * 4;
    g.ticket_bytes = static_cast<uint64_t>(std::min(line, most)) * 8;
  }
  if (g.tt != 32) {
    if (is_mx(mode)) {
      g.atoms = static_cast<int>((mx_sf_cols(mode, K) + 3) / 4);
      g.sf_bytes = static_cast<uint64_t>(g.tiles) * g.atoms * 1024;
    }
    if (gather) g.rows_bytes = static_cast<uint64_t>(R) * row_bytes(mode, K);
  }
  return g;
}

fg_status check_grouped(int mode, int64_t R, int E, int64_t N, int64_t K) {
  const char* what = "fg_grouped_gemm";
  if (!mode_ok(mode)) return fail(FG_ERR_INVALID_ARG, "%s: bad mode %d", what, mode);
  if (E < 1 || E > kMaxExperts) return fail(FG_ERR_SHAPE, "%s: E=%d outside 1..%d", what, E, kMaxExperts);
  if (R < 0 || R > (int64_t(1) << 24)) return fail(FG_ERR_SHAPE, "%s: R=%lld", what, (long long)R);
  if (N <= 0 || N % 128) return fail(FG_ERR_SHAPE, "%s: N=%lld per expert must be a multiple of 128", what, (long long)N);
  if (N > (int64_t(1) << 24)) return fail(FG_ERR_SHAPE, "%s: N=%lld per expert is too large", what, (long long)N);
  return check_nk(mode, N * E, K);
}

}  // namespace

}  // namespace fg

using namespace fg;

extern "C" {

fg_status fg_grouped_gemm_workspace_size(int mode, int64_t R, int E, int64_t N, int64_t K, int gather,
                                         uint64_t* bytes) {
  if (!bytes) return fail(FG_ERR_INVALID_ARG, "null output");
  fg_status s = check_grouped(mode, R, E, N, K);
  if (s != FG_OK) return s;
  *bytes = grouped_plan(mode, R, E, N, K, gather != 0).total();
  return FG_OK;
}

fg_status fg_grouped_gemm(const void* A, const void* a_scales, int64_t T, const int32_t* rows, int64_t R,
                          const int32_t* offsets, int E, const fg_bshuf* b, int mode, void* Y, void* workspace,
                          uint64_t workspace_bytes, uint32_t flags, void* stream) {
  const char* what = "fg_grouped_gemm";
  fg_status s = check_desc(b);
  if (s != FG_OK) return s;
  if (b->mode != mode)
    return fail(FG_ERR_LAYOUT, "%s: weight was preshuffled for %s, call asks for %s", what, mode_name(b->mode), mode_name(mode));
  if (flags & ~FG_FLAG_DEBUG_STALL) return fail(FG_ERR_INVALID_ARG, "%s: unknown flags 0x%x", what, flags);
  if (E < 1 || b->N % E)
    return fail(FG_ERR_SHAPE, "%s: the stacked weight's %lld rows do not divide over E=%d experts", what, (long long)b->N, E);
  const int64_t N = b->N / E, K = b->K;
  if ((s = check_grouped(mode, R, E, N, K)) != FG_OK) return s;
  if (T < 0 || T > (int64_t(1) << 24)) return fail(FG_ERR_SHAPE, "%s: T=%lld", what, (long long)T);
  if (!rows && T < R) return fail(FG_ERR_SHAPE, "%s: A has %lld rows, fewer than R=%lld", what, (long long)T, (long long)R);
  if (R == 0) return FG_OK;
  if (T == 0) return fail(FG_ERR_SHAPE, "%s: no rows of A to gather from", what);
  if (!A || !Y || !offsets) return fail(FG_ERR_INVALID_ARG, "%s: null A, Y or offsets", what);
  if (mode != FG_BF16 && !a_scales) return fail(FG_ERR_INVALID_ARG, "%s: %s needs A scales", what, mode_name(mode));
  if (!aligned(A, 16) || !aligned(Y, 16)) return fail(FG_ERR_ALIGN, "%s: A and Y must be 16-byte aligned", what);
  if (!aligned(offsets, 4) || !aligned(rows, 4) || ((mode == FG_FP8_TENSOR || mode == FG_FP8_BLOCK128) && !aligned(a_scales, 4)))
    return fail(FG_ERR_ALIGN, "%s: offsets, rows and fp32 scales must be 4-byte aligned", what);
  const int64_t rb = row_bytes(mode, K);
  const GroupedPlan g = grouped_plan(mode, R, E, N, K, rows != nullptr, workspace ? workspace_bytes : 0);
  const uint64_t need = g.total();
  if (need) {
    if (!workspace || workspace_bytes < need)
      return fail(FG_ERR_WORKSPACE, "%s: needs a %llu-byte workspace", what, (unsigned long long)need);
    if (!aligned(workspace, 16)) return fail(FG_ERR_ALIGN, "%s: workspace must be 16-byte aligned", what);
  }
  if ((s = check_arch()) != FG_OK) return s;
  GroupedParams p;
  memset(&p, 0, sizeof p);
  p.err = dev_error_ptr();
  if (!p.err) return fail(FG_ERR_CUDA, "device error word unavailable");
  AMaps a_maps;
  CUtensorMap tmap_b;
  memset(&a_maps, 0, sizeof a_maps);
  memset(&tmap_b, 0, sizeof tmap_b);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  uint8_t* a_rows = g.rows_bytes ? ws + g.sf_bytes : nullptr;  // A's rows in the order of Y's
  const bool indexed = rows && !a_rows;
  for (int i = 0; i < (indexed ? 1 : (g.tt == 32 ? 2 : 8)); ++i)
    if ((s = make_tmap(&a_maps.rows[i], a_rows ? a_rows : A, a_rows ? R : T, rb, indexed ? 1 : 16u * (i + 1))) != FG_OK) return s;
  if (mode == FG_MXFP4_FP8A && (s = make_tmap_fp4w(&tmap_b, b->data, b->N, K)) != FG_OK) return s;
  p.b_img = static_cast<const uint8_t*>(b->data);
  p.b_sf = static_cast<const uint8_t*>(b->sf);
  p.b_s = static_cast<const float*>(b->sf);
  p.a_scales = a_scales;
  p.offsets = offsets;
  p.rows = rows;
  p.y = static_cast<__nv_bfloat16*>(Y);
  p.part = reinterpret_cast<float*>(ws);
  p.tickets = reinterpret_cast<unsigned long long*>(ws + g.part_bytes);
  p.epoch = next_epoch() & ((1ull << 48) - 1);
  p.timeout_ns = wait_timeout_ns();
  p.T = static_cast<int>(T);
  p.R = static_cast<int>(R);
  p.E = E;
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.KB = static_cast<int>(rb / 128);
  p.debug_stall = (flags & FG_FLAG_DEBUG_STALL) ? 1 : 0;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  if (g.sf_bytes || g.rows_bytes) {
    PrepParams q{static_cast<const uint8_t*>(A), static_cast<const uint8_t*>(a_scales), offsets, rows, a_rows,
                 g.sf_bytes ? ws : nullptr, p.T, p.R, E, static_cast<int>(rb),
                 is_mx(mode) ? static_cast<int>(mx_sf_cols(mode, K)) : 0, g.atoms, 0};
    if ((e = launch_prep(q, g.tiles, st)) != cudaSuccess) return cuda_fail(e, "grouped product's layout launch");
  }
  if (g.tt == 128) {
    e = launch_grouped_block(a_maps, p, g.blocks, st);
    return e == cudaSuccess ? FG_OK : cuda_fail(e, "grouped product launch");
  }
  if (g.tt == 256) {
    if (g.blocks == 0) return fail(FG_ERR_CUDA, "%s: no room for a pair of SMs", what);
    CUtensorMap tmap_w = tmap_b, tmap_wsf, tmap_asf;
    memset(&tmap_wsf, 0, sizeof tmap_wsf);
    memset(&tmap_asf, 0, sizeof tmap_asf);
    if (mode != FG_MXFP4_FP8A && (s = make_tmap_rows(&tmap_w, b->data, (b->N / 128) * p.KB * 8, 2048, 8)) != FG_OK) return s;
    if (is_mx(mode)) {
      const uint32_t aps = mode == FG_MXFP4 ? 2 : 1;
      if ((s = make_tmap_rows(&tmap_wsf, b->sf, static_cast<int64_t>(b->sf_bytes / 512), 512, aps)) != FG_OK) return s;
      if ((s = make_tmap_rows(&tmap_asf, ws, static_cast<int64_t>(g.sf_bytes / 512), 512, 2 * aps)) != FG_OK) return s;
    }
    e = launch_grouped_pair(mode, a_maps, tmap_w, tmap_wsf, tmap_asf, p, g.blocks, st);
    return e == cudaSuccess ? FG_OK : cuda_fail(e, "grouped product launch");
  }
  switch (mode) {
    case FG_BF16: e = launch_mode<kBF16>(a_maps, tmap_b, p, g.blocks, st); break;
    case FG_FP8_TENSOR: e = launch_mode<kTensor>(a_maps, tmap_b, p, g.blocks, st); break;
    case FG_FP8_BLOCK128: e = launch_mode<kBlock>(a_maps, tmap_b, p, g.blocks, st); break;
    case FG_MXFP8: e = launch_mode<kMXFP8>(a_maps, tmap_b, p, g.blocks, st); break;
    case FG_MXFP4: e = launch_mode<kMXFP4>(a_maps, tmap_b, p, g.blocks, st); break;
    case FG_MXFP8_B32: e = launch_mode<kMXFP8B32>(a_maps, tmap_b, p, g.blocks, st); break;
    case FG_MXFP4_FP8A: e = launch_mode<kMXFP4FP8A>(a_maps, tmap_b, p, g.blocks, st); break;
  }
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "grouped product launch");
}

}  // extern "C"
