// Schedule of the products grouped by expert, from the device's offsets, and the
// parameters of their kernels (fg_grouped.cu has the design).
#pragma once
#include <cuda_bf16.h>

#include "fg_internal.cuh"

namespace fg {

constexpr int kMaxExperts = 1024;
constexpr int kSlabBytes = 16384;  // a 128-row weight tile's K step

// Rows of a token tile come in steps of the MMA's N: 16, or 32 on a pair of SMs
// (TT = 256).
constexpr int tile_step(int tt) { return tt == 256 ? 32 : 16; }

struct GroupedParams {
  const uint8_t* b_img;
  const uint8_t* b_sf;
  const float* b_s;           // FP8_TENSOR: scalar; FP8_BLOCK128: [E * N / 128][K / 128]
  const void* a_scales;
  const int32_t* offsets;     // [E + 1]
  const int32_t* rows;        // [R] or null
  __nv_bfloat16* y;           // [R][N]
  float* part;                // [blocks][2][TT][128] partials (cut line)
  unsigned long long* tickets;  // [blocks] arrivals at the unit that begins last in the block
  unsigned long long epoch;
  uint32_t* err;
  uint64_t timeout_ns;
  int T, R, E, N, K, KB;
  int debug_stall;
};

// A as rows of bytes: boxes of 128 bytes x 16, 32, 48 .. 128 rows, so that a
// tile, or an SM's half of a pair's, is one copy of just its rows (a copy costs
// its issuing warp tens of cycles: 16 boxes of 16 rows a K step held the whole
// kernel back).  Tiles of 32 rows use the first two; with gathered rows the
// first, 1 row high.
struct AMaps {
  CUtensorMap rows[8];
};

// The unit's rows and weight tile.
struct Unit {
  int e, row0, count, nt;
  int width;                    // rows rounded up to the MMA's step
  int tile;                     // token tile, over all experts
};

struct Schedule {
  const int* offs;   // [E + 1] clamped offsets
  const int* tiles;  // [E + 1] token tiles before expert e
  long long units, W, lo, hi;
  int E, NT, KB, blocks, c;
  bool cut;  // the line of all K steps is cut evenly; else units are dealt out whole
};

template <int TT>
__device__ __forceinline__ Unit unit_at(const Schedule& s, long long u) {
  int a = 0, b = s.E;  // the last e with tiles[e] * NT <= u
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (static_cast<long long>(s.tiles[m]) * s.NT <= u) a = m; else b = m;
  }
  const int r = static_cast<int>(u - static_cast<long long>(s.tiles[a]) * s.NT);
  const int n = s.tiles[a + 1] - s.tiles[a];
  const int rows = s.offs[a + 1] - s.offs[a];
  constexpr int STEP = tile_step(TT);
  const int per = ((rows + n - 1) / n + STEP - 1) / STEP * STEP;
  Unit q;
  q.e = a;
  q.nt = r / n;
  const int m = r - q.nt * n;
  q.tile = s.tiles[a] + m;
  q.row0 = s.offs[a] + m * per;
  q.count = min(per, rows - m * per);
  q.width = (q.count + STEP - 1) / STEP * STEP;
  return q;
}

// The unit, known to the compiler as the same in all lanes: what copies and MMAs
// are issued with then stays in uniform registers.
__device__ __forceinline__ Unit uniform(Unit q) {
  q.e = __shfl_sync(0xffffffffu, q.e, 0);
  q.row0 = __shfl_sync(0xffffffffu, q.row0, 0);
  q.count = __shfl_sync(0xffffffffu, q.count, 0);
  q.nt = __shfl_sync(0xffffffffu, q.nt, 0);
  q.width = __shfl_sync(0xffffffffu, q.width, 0);
  q.tile = __shfl_sync(0xffffffffu, q.tile, 0);
  return q;
}

// The offsets, clamped into 0..R, and the token tiles before each expert, by
// the whole block (any count of warps); ends with the block in step.  Offsets
// that decrease would make more tiles than the workspace is laid out for: each
// counts as the largest up to it.
template <int TT>
__device__ __forceinline__ void read_offsets(const int32_t* offsets, int R, int E, int* offs, int* tiles) {
  bool falls = false;
  for (int e = threadIdx.x; e <= E; e += blockDim.x) {
    const int o = min(max(__ldg(offsets + e), 0), R);
    offs[e] = o;
    falls |= e > 0 && min(max(__ldg(offsets + e - 1), 0), R) > o;
  }
  if (__syncthreads_or(falls)) {
    if (threadIdx.x == 0) {
      for (int e = 1; e <= E; ++e) offs[e] = max(offs[e], offs[e - 1]);
    }
    __syncthreads();
  }
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int t = e < E ? (max(0, offs[e + 1] - offs[e]) + TT - 1) / TT : 0;
      int sum = t;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      if (e < E) tiles[e] = carry + sum - t;
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) tiles[E] = carry;
  }
  __syncthreads();
}

// Token tiles of TT = 256 on pairs of SMs.  tmap_w: the weight image as 2 KiB rows
// of 8-byte elements (box: one slab, 8 rows), or fp8 x fp4's blocks; tmap_wsf,
// tmap_asf: the weight's and the tokens' scale images as 512-byte atoms (boxes:
// a slab's atoms).
int grouped_pair_clusters();
cudaError_t launch_grouped_pair(int mode, const AMaps& a_maps, const CUtensorMap& tmap_w, const CUtensorMap& tmap_wsf,
                                const CUtensorMap& tmap_asf, const GroupedParams& p, int ctas, cudaStream_t stream);

}  // namespace fg
