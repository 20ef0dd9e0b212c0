// Column operands: the rows of an activation by expert, transposed and quantised
// along the rows, as the products that sum over rows read them (fg_wgrad.cu).
//
// Places.  Every expert's rows fill slabs of 128 places, the last one's rest is
// zeros; the experts' slabs follow one another and those behind the last expert
// are zeros too.  P places hold R rows of E experts however they fall: 128 for
// every 128 rows, and 128 more for each expert that has a row.
//
// Layout: the weight image and the 32-K scale atoms of an e4m3 matrix [C][P]
// (include/fg.h), one E8M0 per column and 32 places.
#pragma once
#include <cstddef>
#include <cstring>

#include "fg_host.cuh"
#include "fg_ptx.cuh"

namespace fg {

constexpr int kPlaces = 128;       // places of a slab
constexpr int kColumnSlab = 16384;  // its bytes for 128 columns

inline int64_t column_slabs(int64_t R, int64_t E) {
  const int64_t n = R / kPlaces + (E < R ? E : R);
  return n > 0 ? n : 1;
}

// The rows of one slab, and the rows [first, last) that have an expert.
struct SlabRows {
  int row0, count, first, last;
};

// Slab `slab`'s rows by the offsets [E + 1] (null: one expert with all R rows),
// clamped into 0..R; one that decreases counts as the largest before it.  Whole
// warps call it, and each finds the same.
__device__ __forceinline__ SlabRows slab_rows(const int32_t* offsets, int R, int E, int slab) {
  SlabRows q{0, 0, 0, R};
  if (!offsets) {
    q.row0 = slab * kPlaces;
    q.count = min(max(R - q.row0, 0), kPlaces);
    return q;
  }
  const int lane = threadIdx.x & 31;
  int top = min(max(__ldg(offsets), 0), R), slabs = 0;
  bool found = false;
  q.first = top;
  for (int e0 = 0; e0 < E; e0 += 32) {
    int end = e0 + lane < E ? min(max(__ldg(offsets + e0 + lane + 1), 0), R) : 0;
    end = max(end, top);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int o = __shfl_up_sync(0xffffffffu, end, d);
      if (lane >= d) end = max(end, o);
    }
    int start = __shfl_up_sync(0xffffffffu, end, 1);
    start = lane == 0 ? top : start;
    if (!found) {
      const int n = (end - start + kPlaces - 1) / kPlaces;
      int sum = n;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int o = __shfl_up_sync(0xffffffffu, sum, d);
        if (lane >= d) sum += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, slabs + sum > slab);
      if (past) {
        const int src = __ffs(past) - 1;
        const int before = slabs + __shfl_sync(0xffffffffu, sum - n, src);
        q.row0 = __shfl_sync(0xffffffffu, start, src) + (slab - before) * kPlaces;
        q.count = min(__shfl_sync(0xffffffffu, end, src) - q.row0, kPlaces);
        found = true;
      }
      slabs += __shfl_sync(0xffffffffu, sum, 31);
    }
    top = __shfl_sync(0xffffffffu, end, 31);
  }
  q.last = top;
  return q;
}

// The clamped offsets offs[0..E] and the slabs before each expert, slabs[0..E], by
// one warp (offsets null: one expert with all R rows); never more than `most` slabs.
__device__ __forceinline__ void read_slabs(const int32_t* offsets, int R, int E, int most, int* offs, int* slabs) {
  const int lane = threadIdx.x & 31;
  if (!offsets) {
    if (lane < 2) {
      offs[lane] = lane * R;
      slabs[lane] = lane * min((R + kPlaces - 1) / kPlaces, most);
    }
    return;
  }
  int top = 0, before_all = 0;
  for (int e0 = 0; e0 <= E; e0 += 32) {
    const int e = e0 + lane;
    int o = e <= E ? min(max(__ldg(offsets + e), 0), R) : 0;
    o = max(o, top);
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, o, d);
      if (lane >= d) o = max(o, x);
    }
    int before = __shfl_up_sync(0xffffffffu, o, 1);
    if (lane == 0) before = e0 == 0 ? o : top;
    int sum = (o - before + kPlaces - 1) / kPlaces;  // of expert e - 1
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, sum, d);
      if (lane >= d) sum += x;
    }
    if (e <= E) {
      offs[e] = o;
      slabs[e] = min(before_all + sum, most);
    }
    top = __shfl_sync(0xffffffffu, o, 31);
    before_all += __shfl_sync(0xffffffffu, sum, 31);
  }
}

// Descriptor of a column operand with C columns and P places.
inline void column_descriptor(int64_t C, int64_t P, void* data, void* sf, fg_bshuf* out) {
  fg_bshuf d;
  memset(&d, 0, sizeof d);
  d.magic = FG_BSHUF_MAGIC;
  d.version = FG_BSHUF_VERSION;
  d.mode = FG_MXFP8_B32;
  d.tile_rows = 128;
  d.N = C;
  d.K = P;
  d.data = data;
  d.sf = sf;
  d.data_bytes = static_cast<uint64_t>(C) * P;
  d.sf_bytes = static_cast<uint64_t>(C) * P / 32;
  // the check word as check_desc knows it: FNV-1a of the fields before it
  uint64_t h = 1469598103934665603ull;
  const uint8_t* b = reinterpret_cast<const uint8_t*>(&d);
  for (size_t i = 0; i < offsetof(fg_bshuf, check); ++i) h = (h ^ b[i]) * 1099511628211ull;
  d.check = h ^ 0x5eedf00dcafe1234ull;
  *out = d;
}

// C columns and R rows of E experts within a column operand's limits.
fg_status check_columns(const char* what, int64_t C, int64_t R, int E);

}  // namespace fg
