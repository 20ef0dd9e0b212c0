// What the backward pass of an 8-bit layer lays out: weights in 128 x 128 blocks,
// as they are or transposed; activations as column operands (fg_columns.cuh); and
// the gated activation's gradient from its 8-bit checkpoint, which leaves both
// forms at once.
//
// Squares.  A warp takes 32 rows x 32 columns: thread (tl, fl) = (lane / 4, lane %
// 4) rows 4 tl .. + 3 and columns 8 fl .. + 7.  A block of 32 values along either
// side then lies in one warp.  Its largest magnitude is found by halves: in each
// exchange a lane gives away the candidates of the half that it does not keep, so
// seven shuffles leave one column's maximum in each lane (three for rows), and
// the scale is worked out once, not by every lane.  Eight values along a row are
// eight bytes of codes, four along a column one word of the transposed image: the
// transposition costs nothing, the pairs of values that are rounded together are
// only others.  All stores fill whole 32-byte sectors.
#include <cuda_bf16.h>

#include <algorithm>

#include "fg_columns.cuh"
#include "fg_internal.cuh"
#include "fg_values.cuh"

namespace fg {

namespace {

constexpr int kMaxExperts = 1024;
constexpr int kMaxTopK = 32;
constexpr int kWide = 128;    // columns of a block of threads: four squares side by side
constexpr int kThreads = 128;

struct Square {  // a thread's part of one: rows i, columns 2 q and 2 q + 1
  Pair p[4][4];
};

// ------------------------------------------------------------------ inputs

enum Format { kF32Rows, kBf16Rows, kE8m0By32, kE8m0By128, kF32By128 };

struct Source {
  const void* x;
  const void* scales;
  int64_t ld;    // elements from row to row
  int64_t cols;
};

// What eight codes and their scale stand for.
__device__ __forceinline__ void decode(uint2 codes, float scale, Pair (&v)[4]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 f = e4m3_values((q < 2 ? codes.x : codes.y) >> (16 * (q & 1)));
    v[q] = mul(pair_of(f.x, f.y), pair_of(scale, scale));
  }
}

// Eight consecutive values of a row on their way.
constexpr int scale_block(int fmt) { return fmt == kE8m0By32 ? 32 : 128; }

template <int FMT>
struct Eight {
  static constexpr int BYTES = 1;  // of a value
  uint2 codes;
  uint32_t scale;  // as it lies in memory: worked out here, it would be waited for
  __device__ __forceinline__ void load(uintptr_t row, uintptr_t scales, int col) {
    codes = __ldcs(reinterpret_cast<const uint2*>(row + col));
    if (FMT == kF32By128) scale = __ldg(reinterpret_cast<const uint32_t*>(scales) + col / scale_block(FMT));
    else scale = __ldg(reinterpret_cast<const uint8_t*>(scales) + col / scale_block(FMT));
  }
  __device__ __forceinline__ void zero() {
    codes = make_uint2(0, 0);
    scale = 0;
  }
  __device__ __forceinline__ void widen(Pair (&v)[4]) const {
    decode(codes, FMT == kF32By128 ? __uint_as_float(scale) : e8m0_up(scale), v);
  }
};

template <typename T>
struct PlainEight {
  static constexpr int BYTES = sizeof(T);
  Raw8<T> raw;
  __device__ __forceinline__ void load(uintptr_t row, uintptr_t, int col) { raw.load_once(reinterpret_cast<const T*>(row) + col); }
  __device__ __forceinline__ void zero() { raw.zero(); }
  __device__ __forceinline__ void widen(Pair (&v)[4]) const {
    float f[8];
    raw.widen(f);
#pragma unroll
    for (int q = 0; q < 4; ++q) v[q] = pair_of(f[2 * q], f[2 * q + 1]);
  }
};

template <>
struct Eight<kBf16Rows> : PlainEight<__nv_bfloat16> {};
template <>
struct Eight<kF32Rows> : PlainEight<float> {};

// ----------------------------------------------------------- column stores

struct Image {
  uint8_t* data;  // null: not wanted
  uint8_t* sf;
  int slabs;      // of a row of 128 columns
};

// One exchange by halves: of the candidates m[0 .. 2 n) a lane keeps the first n,
// or with bit `bit` of its index the others.
template <int N>
__device__ __forceinline__ void halve(uint32_t* m, int bit) {
  const bool upper = (threadIdx.x & bit) != 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t give = upper ? m[j] : m[j + N], keep = upper ? m[j + N] : m[j];
    m[j] = max(keep, __shfl_xor_sync(0xffffffffu, give, bit));
  }
}

// Where this lane's eight columns begin in slab `slab` of an image: columns f0 + 8 (lane
// % 4), places 4 (lane / 4).  16-byte piece i of a column's places lies at i ^ (column %
// 8), which is 0 for the first of the eight.
__device__ __forceinline__ uintptr_t lane_place(const Image& im, int f0, int slab) {
  const int lane = threadIdx.x & 31;
  return reinterpret_cast<uintptr_t>(im.data) + (static_cast<size_t>(f0 >> 7) * im.slabs + slab) * kColumnSlab + (f0 & 127) * 128 +
         (lane & 3) * 1024 + (lane >> 2) * 4;
}

// The warp's square as 32 columns x 32 places, the places 32 b .. of the slab that
// `place` is lane_place() of.  The scale's byte goes into byte b of `word`, for the
// column that this lane keeps.
__device__ __forceinline__ void store_columns(const Square& v, uintptr_t place, int b, uint32_t& word) {
  const int fl = threadIdx.x & 3;
  uint32_t m[8];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float2 x[4] = {halves(v.p[0][q]), halves(v.p[1][q]), halves(v.p[2][q]), halves(v.p[3][q])};
    m[2 * q] = __float_as_uint(largest(largest(x[0].x, x[1].x, x[2].x), x[3].x, x[3].x));
    m[2 * q + 1] = __float_as_uint(largest(largest(x[0].y, x[1].y, x[2].y), x[3].y, x[3].y));
  }
  halve<4>(m, 16);
  halve<2>(m, 8);
  halve<1>(m, 4);
  const bool finite = m[0] < 0x7f800000u;
  const int c = finite ? e8m0_of(m[0]) : 255;
  word |= static_cast<uint32_t>(c) << (8 * b);
  const float mine = e8m0_down(finite ? c : 127);
  const bool whole = __all_sync(0xffffffffu, finite);
  const uintptr_t out = place + b * 32;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    // the lane that kept column j: bits 16, 8, 4 of its index are those of j
    const int owner = ((q & 2) << 3) | ((q & 1) << 3) | fl;
    const Pair f = pair_of(__shfl_sync(0xffffffffu, mine, owner), __shfl_sync(0xffffffffu, mine, owner | 4));
    float2 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = halves(mul(v.p[i][q], f));
    if (!whole) {
      const bool lo = __shfl_sync(0xffffffffu, static_cast<int>(finite), owner) != 0;
      const bool hi = __shfl_sync(0xffffffffu, static_cast<int>(finite), owner | 4) != 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = make_float2(lo ? x[i].x : 0.f, hi ? x[i].y : 0.f);
    }
    *reinterpret_cast<uint32_t*>((out ^ (2 * q * 16)) + 2 * q * 128) =
        e4m3x2(x[0].x, x[1].x) | (e4m3x2(x[2].x, x[3].x) << 16);
    *reinterpret_cast<uint32_t*>((out ^ ((2 * q + 1) * 16)) + (2 * q + 1) * 128) =
        e4m3x2(x[0].y, x[1].y) | (e4m3x2(x[2].y, x[3].y) << 16);
  }
}

// 32 places of zeros.
__device__ __forceinline__ void store_no_columns(const Image& im, int f0, int slab, int b, uint32_t& word) {
  const int lane = threadIdx.x & 31;
  uint8_t* out = im.data + (static_cast<size_t>(f0 >> 7) * im.slabs + slab) * kColumnSlab + (f0 & 127) * 128;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = 16 * h + (lane >> 1), piece = 2 * b + (lane & 1);
    *reinterpret_cast<uint4*>(out + row * 128 + ((piece ^ (row & 7)) << 4)) = make_uint4(0, 0, 0, 0);
  }
  word |= 127u << (8 * b);
}

// The scales of the column that this lane kept: a slab's four blocks of places, or
// (parts = 4) block b's alone.
__device__ __forceinline__ void store_atoms(const Image& im, int f0, int slab, int parts, int b, uint32_t word) {
  const int lane = threadIdx.x & 31;
  const int j = ((lane >> 4) & 1) * 4 + ((lane >> 3) & 1) * 2 + ((lane >> 2) & 1);
  const int f = f0 + (lane & 3) * 8 + j;
  uint8_t* atom = im.sf + (static_cast<size_t>(f >> 7) * im.slabs + slab) * 512 + 16 * (f & 31) + 4 * ((f & 127) >> 5);
  if (parts == 1) *reinterpret_cast<uint32_t*>(atom) = word;
  else atom[b] = static_cast<uint8_t>(word >> (8 * b));
}

// ------------------------------------------------------- quantise to columns

struct ColumnsParams {
  Source in;
  const int32_t* offsets;
  const int32_t* rows;  // null: row i itself
  Image image;
  int T, R, E;
};

// A block of threads takes one slab's 128 places, or where blocks would be few 32 of
// them, and every gridDim.x-th tile of 128 columns: the rows' places are found once.
// 32 places at a time, the next ones' values asked for before these are worked on.
// 32768 x 4096 bf16 in 68 us (6.0 TB/s), 32768 rows of 7168 codes gathered from 4096 in
// 113, whose 12 instructions a value take 71.
template <int FMT>
__global__ void __launch_bounds__(kThreads) columns_kernel(const ColumnsParams p) {
  // the places' rows and their scales; none: null
  __shared__ __align__(16) uintptr_t row_sh[kPlaces], scale_sh[kPlaces];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tl = lane >> 2, fl = lane & 3;
  const int slab = blockIdx.y, span = 4 / gridDim.z, b0 = blockIdx.z * span;
  const int tiles = static_cast<int>(p.in.cols / kWide);
  const SlabRows q = slab_rows(p.offsets, p.R, p.E, slab);
  const int squares = min(max((q.count + 31) / 32 - b0, 0), span);  // with a row, of this block's
  {
    uintptr_t x = 0, scales = 0;
    if (threadIdx.x < q.count) {
      int64_t row = q.row0 + threadIdx.x;
      if (p.rows) row = min(max(__ldg(p.rows + row), 0), p.T - 1);
      x = reinterpret_cast<uintptr_t>(p.in.x) + row * p.in.ld * Eight<FMT>::BYTES;
      scales = reinterpret_cast<uintptr_t>(p.in.scales) + row * (p.in.cols / scale_block(FMT)) * (FMT == kF32By128 ? 4 : 1);
    }
    row_sh[threadIdx.x] = x;
    scale_sh[threadIdx.x] = scales;
  }
  __syncthreads();
  Eight<FMT> next[4];
  // the values of square n: places 32 (b0 + n % squares), column tile n / squares of the block's
  const int count = squares * ((tiles - static_cast<int>(blockIdx.x) + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
  int ask_b = 0, ask_col = blockIdx.x * kWide + warp * 32 + fl * 8;
  auto ask = [&] {
    const int at = 32 * (b0 + ask_b) + 4 * tl;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uintptr_t row = row_sh[at + i];
      next[i].zero();
      if (row) next[i].load(row, scale_sh[at + i], ask_col);
    }
    if (++ask_b == squares) {
      ask_b = 0;
      ask_col += gridDim.x * kWide;
    }
  };
  if (count > 0) ask();
  int n = 0;
  uintptr_t place = lane_place(p.image, blockIdx.x * kWide + warp * 32, slab);
#pragma unroll 1
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int f0 = tile * kWide + warp * 32;
    uint32_t word = 0;
#pragma unroll 1
    for (int b = 0; b < squares; ++b) {
      Square v;
#pragma unroll
      for (int i = 0; i < 4; ++i) next[i].widen(v.p[i]);
      if (++n < count) ask();
      store_columns(v, place, b0 + b, word);
    }
    place += static_cast<size_t>(gridDim.x) * p.image.slabs * kColumnSlab;
    for (int b = squares; b < span; ++b) store_no_columns(p.image, f0, slab, b0 + b, word);
    store_atoms(p.image, f0, slab, gridDim.z, b0, word);
  }
}

// ------------------------------------------------ gated activation, backward

struct SwigluParams {
  Source dy;              // [R][K]
  Source saved;           // [R][2 K]
  const float* weights;   // [T][k] (null: none)
  const int32_t* rows;    // [R]
  const int32_t* slots;   // [T][k]
  const int32_t* offsets;
  uint8_t* codes;         // [R][2 K]
  void* scales;
  void* dx;               // [R][2 K] (null: not wanted)
  float* dots;            // [R][dot_parts]: sums over 32 columns each (weights given)
  Image dx_image, act_image;
  int T, R, E, K, k, dot_parts;
};

// Codes and scales of the warp's square along its rows, `rows` of them.  out: where
// this lane's eight codes of its first row go, `cols` bytes from row to row; block: the
// first row's scale block.  Scale blocks of 128 take the maximum over the four warps,
// through `part` [4][32].
template <int FMT>
__device__ __forceinline__ void store_rows(const Square& v, uint8_t* out, int64_t cols, void* scales, int64_t block, int rows,
                                           uint32_t (*part)[32]) {
  const int lane = threadIdx.x & 31, tl = lane >> 2;
  uint32_t m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x[4] = {halves(v.p[i][0]), halves(v.p[i][1]), halves(v.p[i][2]), halves(v.p[i][3])};
    m[i] = __float_as_uint(largest(largest(largest(x[0].x, x[0].y, x[1].x), x[1].y, x[2].x), largest(x[2].y, x[3].x, x[3].y), 0.f));
  }
  halve<2>(m, 1);
  halve<1>(m, 2);
  const int keep = ((lane & 1) << 1) | ((lane >> 1) & 1);  // row 4 tl + keep's maximum is here
  const int mine = 4 * tl + keep;
  if (FMT != kE8m0By32) {
    part[threadIdx.x >> 5][mine] = m[0];
    __syncthreads();
    m[0] = max(max(part[0][mine], part[1][mine]), max(part[2][mine], part[3][mine]));
  }
  const bool finite = m[0] < 0x7f800000u;
  const int64_t at = block + mine * (cols / scale_block(FMT));
  const bool stores = mine < rows && (FMT == kE8m0By32 || threadIdx.x < 32);
  float scale;  // what values are multiplied by (E8M0) or divided by (with their signs turned: see Over)
  if (FMT == kF32By128) {
    scale = f32_scale_of(finite ? m[0] : 0u);
    if (stores) static_cast<float*>(scales)[at] = finite ? scale : __uint_as_float(0x7fc00000u);
  } else {
    const int c = finite ? e8m0_of(m[0]) : 127;
    scale = e8m0_down(c);
    if (stores) static_cast<uint8_t*>(scales)[at] = static_cast<uint8_t>(finite ? c : 255);
  }
  const bool whole = __all_sync(0xffffffffu, finite);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int owner = (lane & ~3) | ((i >> 1) & 1) | ((i & 1) << 1);
    const float f = __shfl_sync(0xffffffffu, scale, owner);
    const bool ok = whole || __shfl_sync(0xffffffffu, static_cast<int>(finite), owner) != 0;
    uint32_t w[4];
    if constexpr (FMT == kF32By128) {
      const Over over(f);
      if (whole && over.sure) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 x = halves(over(v.p[i][q]));
          w[q] = e4m3x2(x.x, x.y);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float2 x = halves(v.p[i][q]);
          w[q] = e4m3x2(ok ? __fdiv_rn(-x.x, f) : -0.f, ok ? __fdiv_rn(-x.y, f) : -0.f);
        }
      }
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float2 x = halves(mul(v.p[i][q], pair_of(f, f)));
        if (!whole) x = make_float2(ok ? x.x : 0.f, ok ? x.y : 0.f);
        w[q] = e4m3x2(x.x, x.y);
      }
    }
    constexpr uint32_t TURN = FMT == kF32By128 ? kMinusCodes : 0u;
    const uint2 o = make_uint2((w[0] | (w[1] << 16)) ^ TURN, (w[2] | (w[3] << 16)) ^ TURN);
    if (4 * tl + i < rows) *reinterpret_cast<uint2*>(out + i * cols) = o;
  }
}

// What a thread's loads for one square have landed in: its own bytes alone, so that
// nobody waits for another.
template <typename T>
struct Landing {
  uint4 dy[4][sizeof(T) / 2][kThreads];
  uint2 g[4][kThreads], u[4][kThreads];
};

// 16 or 8 bytes to shared memory, zeros where there are none to read.
__device__ __forceinline__ void fetch16(void* dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void fetch8(void* dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 8 : 0) : "memory");
}

// With g, u the checkpoint's values, s = sigmoid(g) and w the row's routing weight:
//   act = g s u,  dots = sum dy act,  dg = w dy u s (1 + g (1 - s)),  du = w dy g s.
// e = exp(-g), held below 2^128, and s = 1 / (1 + e) come from the fast power and
// reciprocal (2 ulp and 1 ulp), so s is 0 below g = -87.3, where it is under 2^-126.  The
// exponent -g log2(e) is off by its own rounding and the constant's, together 1.22 * 2^-24
// of itself, and so e by 1.22 |g| 2^-24 more: s is within (8 + 1.3 |g|) 2^-24 of itself for
// negative g, within 8 * 2^-24 for others, whose e is the smaller part of 1 + e.  g (1 - s)
// is g s e, without the cancellation of 1 - s that a large g would multiply.
//
// A block of threads takes one slab's 128 rows x 128 columns at a time, 32 rows in
// turn, and asks for the next 32 rows' bytes before it works on these: with four
// blocks an SM, whose registers they fill, nothing else covers the loads.  32760 x
// 2048 with columns in 192 us, where its bytes take 91: some 60 instructions for each value
// of the activation, whose three results are each rounded twice, along rows and along
// columns, and 54 % of the issue slots used by the four warps that their registers leave a
// scheduler.  371 with loads that are waited for and values one by one
// instead of in pairs, 208 with addresses worked out for each.  Blocks of threads that
// stay and take several slabs spill: 321; so do two results' exchanges side by side: 236.
template <int FMT, typename T>
__global__ void __launch_bounds__(kThreads, 4) swiglu_backward_kernel(const SwigluParams p) {
  __shared__ uint32_t part[2][2][4][32];
  __shared__ float weight_sh[kPlaces];
  extern __shared__ uint8_t landing_sh[];
  Landing<T>* landing = reinterpret_cast<Landing<T>*>(landing_sh);
  pdl_wait();
  pdl_launch_dependents();
  constexpr int S = scale_block(FMT);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, tl = lane >> 2, fl = lane & 3;
  const int slab = blockIdx.y, tiles = (p.K + kWide - 1) / kWide;
  const int64_t cols = 2 * static_cast<int64_t>(p.K);
  const SlabRows q = slab_rows(p.offsets, p.R, p.E, slab);
  const int span = 4 / gridDim.z, b0 = blockIdx.z * span;             // squares of this block, and the first
  const int squares = min(max((q.count + 31) / 32 - b0, 0), span);   // ... that have a row
  // The next square: rows 32 next_b of the slab, column tile next_tile.  The
  // checkpoint's scales of its row `lane` as they lie in memory, and its bytes.
  int next_b = b0, next_tile = blockIdx.x;
  uint32_t gs_next = 0, us_next = 0;
  auto ask = [&](int stage) {
    const int f0 = next_tile * kWide + warp * 32;
    // (32-blocks: the last warps may have no columns)
    const int mine = f0 < p.K ? q.count - 32 * next_b - 4 * tl : 0;  // rows from this lane's first
    const int64_t row = q.row0 + 32 * next_b + 4 * tl;
    const int c = f0 + fl * 8;
    const T* dy = static_cast<const T*>(p.dy.x) + row * p.dy.ld + c;
    const uint8_t* saved = static_cast<const uint8_t*>(p.saved.x) + row * cols + c;
    Landing<T>& to = landing[stage];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h)
        fetch16(&to.dy[i][h][tid], dy + i * p.dy.ld + 8 * h / static_cast<int>(sizeof(T) / 2), i < mine);
      fetch8(&to.g[i][tid], saved + i * cols, i < mine);
      fetch8(&to.u[i][tid], saved + i * cols + p.K, i < mine);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto ask_scales = [&] {
    const int f0 = next_tile * kWide + warp * 32;
    gs_next = us_next = 0;  // (rows that are not there have codes 0)
    if (f0 < p.K && 32 * next_b + lane < q.count) {
      const int64_t at = (q.row0 + 32 * next_b + lane) * (cols / S) + f0 / S;
      if (FMT == kF32By128) {
        gs_next = __ldg(static_cast<const uint32_t*>(p.saved.scales) + at);
        us_next = __ldg(static_cast<const uint32_t*>(p.saved.scales) + at + p.K / S);
      } else {
        gs_next = __ldg(static_cast<const uint8_t*>(p.saved.scales) + at);
        us_next = __ldg(static_cast<const uint8_t*>(p.saved.scales) + at + p.K / S);
      }
    }
  };
  // zeros in the block's squares from r on, and all their scales
  auto close = [&](int f0, int r, uint32_t g, uint32_t u, uint32_t a) {
    for (; r < b0 + span; ++r) {
      store_no_columns(p.dx_image, f0, slab, r, g);
      store_no_columns(p.dx_image, p.K + f0, slab, r, u);
      store_no_columns(p.act_image, f0, slab, r, a);
    }
    store_atoms(p.dx_image, f0, slab, gridDim.z, b0, g);
    store_atoms(p.dx_image, p.K + f0, slab, gridDim.z, b0, u);
    store_atoms(p.act_image, f0, slab, gridDim.z, b0, a);
  };
  if (squares > 0) {
    ask(0);
    ask_scales();
    // meanwhile the slab's routing weights: a row's is that of the choice whose slot it is
    float w = 1.f;
    if (p.weights) {
      w = 0.f;
      if (tid < q.count) {
        const int64_t t = min(max(__ldg(p.rows + q.row0 + tid), 0), p.T - 1);
        for (int j0 = 0; j0 < p.k; j0 += 8) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j0 + j < p.k && __ldg(p.slots + t * p.k + j0 + j) == q.row0 + tid) w = __ldg(p.weights + t * p.k + j0 + j);
        }
      }
    }
    weight_sh[tid] = w;
  }
  __syncthreads();
  int stage = 0;
#pragma unroll 1
  for (int tile = blockIdx.x; squares > 0 && tile < tiles; tile += gridDim.x) {
    const int f0 = tile * kWide + warp * 32;
    const bool inside = f0 < p.K;
    uint32_t word_g = 0, word_u = 0, word_a = 0;
#pragma unroll 1
    for (int b = b0; b < b0 + squares; ++b, stage ^= 1) {
      const uint32_t gs_row = gs_next, us_row = us_next;
      if (++next_b == b0 + squares) {
        next_b = b0;
        next_tile += gridDim.x;
      }
      const bool more = next_tile < tiles;
      if (more) {
        ask(stage ^ 1);
        asm volatile("cp.async.wait_group 1;" ::: "memory");
      } else {
        asm volatile("cp.async.wait_group 0;" ::: "memory");
      }
      const Landing<T>& from = landing[stage];
      auto scale = [](uint32_t x) { return FMT == kF32By128 ? __uint_as_float(x) : e8m0_up(x); };
      const int64_t row0 = q.row0 + 32 * b;
      const int rows = q.count - 32 * b;
      Square act, dg, du;
      float dot[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float w = weight_sh[32 * b + 4 * tl + i];
        const float gs = scale(__shfl_sync(0xffffffffu, gs_row, 4 * tl + i)), us = scale(__shfl_sync(0xffffffffu, us_row, 4 * tl + i));
        Pair g[4], u[4], dy[4];
        decode(from.g[i][tid], gs, g);
        decode(from.u[i][tid], us, u);
        Eight<sizeof(T) == 2 ? kBf16Rows : kF32Rows> raw;
#pragma unroll
        for (int h = 0; h < static_cast<int>(sizeof(T) / 2); ++h) raw.raw.q[h] = from.dy[i][h][tid];
        raw.widen(dy);
        Pair sum = pair_of(0.f, 0.f);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          constexpr float kLog2e = 1.44269504088896341f;
          float2 e = halves(mul(g[c], pair_of(-kLog2e, -kLog2e)));
          e = make_float2(fminf(e.x, 127.9f), fminf(e.y, 127.9f));  // (a NaN is in g too)
          asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
          asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
          const Pair ee = pair_of(e.x, e.y), one = pair_of(1.f, 1.f);
          float2 h = halves(add(ee, one));
          asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(h.x));
          asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(h.y));
          const Pair sg = pair_of(h.x, h.y), gs_ = mul(g[c], sg), up = fma(gs_, ee, one);  // up: 1 + g (1 - s)
          const Pair a = mul(gs_, u[c]), d = mul(dy[c], pair_of(w, w));
          sum = fma(dy[c], a, sum);
          act.p[i][c] = mul(a, pair_of(w, w));
          dg.p[i][c] = mul(d, mul(u[c], mul(sg, up)));  // (no product larger than its result but by rounding)
          du.p[i][c] = mul(d, gs_);
        }
        const float2 s = halves(sum);
        dot[i] = s.x + s.y;
      }
      if (p.dots) {
        // by halves, as the maxima: each lane keeps one row's sum over its eight columns x four
        const bool odd = (lane & 1) != 0, upper = (lane & 2) != 0;
        const float x = (odd ? dot[2] : dot[0]) + __shfl_xor_sync(0xffffffffu, odd ? dot[0] : dot[2], 1);
        const float y = (odd ? dot[3] : dot[1]) + __shfl_xor_sync(0xffffffffu, odd ? dot[1] : dot[3], 1);
        const float z = (upper ? y : x) + __shfl_xor_sync(0xffffffffu, upper ? x : y, 2);
        const int mine = 4 * tl + 2 * (lane & 1) + ((lane >> 1) & 1);
        if (inside && mine < rows) p.dots[(row0 + mine) * p.dot_parts + tile * 4 + warp] = z;
      }
      if (inside && p.dx_image.data) store_columns(act, lane_place(p.act_image, f0, slab), b, word_a);
      // Only now, with the activation's values gone: scales asked for together with the
      // rows would live in registers that there are none of, and spilling them waits
      // for the load.
      if (more) ask_scales();
      if (!inside) continue;
      if (p.dx_image.data) {
        store_columns(dg, lane_place(p.dx_image, f0, slab), b, word_g);
        store_columns(du, lane_place(p.dx_image, p.K + f0, slab), b, word_u);
        if (b + 1 == b0 + squares) close(f0, b + 1, word_g, word_u, word_a);
      }
      const int64_t out = (row0 + 4 * tl) * cols + f0 + fl * 8, block = row0 * (cols / S) + f0 / S;
      store_rows<FMT>(dg, p.codes + out, cols, p.scales, block, rows, part[stage][0]);
      store_rows<FMT>(du, p.codes + out + p.K, cols, p.scales, block + p.K / S, rows, part[stage][1]);
      if (p.dx) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (4 * tl + i < rows) {
            T* to = static_cast<T*>(p.dx) + out + i * cols;
            float x[8], y[8];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              *reinterpret_cast<float2*>(&x[2 * c]) = halves(dg.p[i][c]);
              *reinterpret_cast<float2*>(&y[2 * c]) = halves(du.p[i][c]);
            }
            store8(to, x);
            store8(to + p.K, y);
          }
        }
      }
    }
  }
  // Rows that no expert has: zeros.  The slabs are more than the rows / 128, so
  // that each takes its 128 of them.  And squares without rows are zeros.
  const int none = q.first + (p.R - q.last);
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    if (squares == 0 && p.dx_image.data) close(tile * kWide + warp * 32, b0, 0, 0, 0);
    if (b0 > 0) continue;
    for (int i = slab * kPlaces + warp; i < min(none, (slab + 1) * kPlaces); i += 4) {
      const int64_t row = i < q.first ? i : q.last + (i - q.first);
      const int c = tile * kWide + lane * 4;
      if (p.dots && lane < 4 && tile * 4 + lane < p.dot_parts) p.dots[row * p.dot_parts + tile * 4 + lane] = 0.f;
      if (c >= p.K) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t at = row * cols + h * static_cast<int64_t>(p.K) + c;
        *reinterpret_cast<uint32_t*>(p.codes + at) = 0u;
        if (p.dx) {
#pragma unroll
          for (int j = 0; j < 4; ++j) static_cast<T*>(p.dx)[at + j] = T(0.f);
        }
        if (c % S == 0) {
          if (FMT == kF32By128) static_cast<float*>(p.scales)[at / 128] = 1.f;
          else static_cast<uint8_t*>(p.scales)[at / S] = 127;
        }
      }
    }
  }
}

// dweights[t][j] = the sum of the partial dots of its slot's row, always in the same
// order; 0 where there is no choice.  Eight threads a choice, so that they read whole
// sectors.
__global__ void __launch_bounds__(256) dweights_kernel(const float* __restrict__ dots, const int32_t* __restrict__ slots,
                                                       int64_t choices, int R, int parts, float* __restrict__ dweights) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 8) + threadIdx.x / 8;
  const int slot = i < choices ? __ldg(slots + i) : -1;
  float sum = 0.f;
  if (slot >= 0 && slot < R) {
    const float* d = dots + static_cast<size_t>(slot) * parts;
#pragma unroll 8
    for (int x = threadIdx.x & 7; x < parts; x += 8) sum += __ldcg(d + x);
  }
#pragma unroll
  for (int d = 4; d > 0; d /= 2) sum += __shfl_xor_sync(0xffffffffu, sum, d);
  if (i < choices && (threadIdx.x & 7) == 0) dweights[i] = sum;
}

// ------------------------------------------------------------------ weights

// 128 x 128 blocks of weights: scale and codes, straight or transposed, by 16 warps, a
// square each, so that the values wait for the block's maximum in registers.  Blocks of
// threads stay and take every gridDim.x-th block of the weights; the next one's bytes
// are on their way to shared memory meanwhile.  8 weights of 4096 x
// 7168 bf16, transposed, in 110 us (6.4 TB/s, 0.94 of a copy's rate); 150 with a block of
// threads for each block of weights and a division for each value.
constexpr int kWeightThreads = 512;

template <typename T, bool TRANSPOSE>
__global__ void __launch_bounds__(kWeightThreads, 2) weight_kernel(const T* __restrict__ w, int64_t ld, int64_t stride, int N, int K,
                                                                   int blocks, uint8_t* __restrict__ codes,
                                                                   float* __restrict__ scales) {
  constexpr int Q = sizeof(T) / 2;  // 16-byte pieces of eight values
  extern __shared__ uint8_t landing_sh[];
  auto landing = reinterpret_cast<uint4(*)[4][Q][kWeightThreads]>(landing_sh);
  __shared__ uint32_t part[2][16];
  pdl_wait();
  pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, tl = lane >> 2, fl = lane & 3;
  const int KB = K / 128, NB = N / 128;
  struct At {
    int e, n, k;
  };
  auto place = [&](int b) {  // block b's weight and first row and column, in blocks
    At a;
    const int row = b / KB;
    a.k = b - row * KB;
    a.e = row / NB;
    a.n = row - a.e * NB;
    return a;
  };
  const int in_n = 32 * (warp >> 2) + 4 * tl, in_k = 32 * (warp & 3) + 8 * fl;
  // Four lanes fetch neighbouring pieces, so that an instruction takes whole sectors, also
  // where a lane's eight values are two pieces: fp32 weights of the size above in 272 us
  // straight and 268 transposed; 273 and 292 with each lane fetching its own.
  auto ask = [&](const At& a, int stage) {
    const T* src = w + a.e * stride + (a.n * 128 + in_n) * ld + a.k * 128 + 32 * (warp & 3);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int h = 0; h < Q; ++h) {
        const int piece = 4 * h + fl;
        fetch16(&landing[stage][i][piece % Q][threadIdx.x - fl + piece / Q], src + i * ld + piece * (8 / Q), true);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  At next = place(blockIdx.x);
  ask(next, 0);
  int stage = 0;
#pragma unroll 1
  for (int b = blockIdx.x; b < blocks; b += gridDim.x, stage ^= 1) {
    const At a = next;
    if (b + static_cast<int>(gridDim.x) < blocks) {
      next = place(b + gridDim.x);
      ask(next, stage ^ 1);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    } else {
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    }
    __syncwarp();
    const int64_t e = a.e;
    const int n = a.n * 128 + in_n, k = a.k * 128 + in_k;
    float v[4][8], most = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      Raw8<T> raw;
#pragma unroll
      for (int h = 0; h < Q; ++h) raw.q[h] = landing[stage][i][h][threadIdx.x];
      raw.widen(v[i]);
#pragma unroll
      for (int j = 0; j < 8; j += 2) most = largest(most, v[i][j], v[i][j + 1]);
    }
    uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
    if (lane == 0) part[stage][warp] = top;
    __syncthreads();
    top = __reduce_max_sync(0xffffffffu, part[stage][lane & 15]);
    const bool finite = top < 0x7f800000u;
    const float s = f32_scale_of(finite ? top : 0u);
    if (threadIdx.x == 0) {
      const int64_t at = TRANSPOSE ? (e * KB + a.k) * NB + a.n : (e * NB + a.n) * KB + a.k;
      scales[at] = finite ? s : __uint_as_float(0x7fc00000u);
    }
    const Over over(s);
    // words of four codes: column j's, or (row i, half) 2 i + half
    uint32_t c[8];
    auto words = [&](auto quotient) {  // the negative one of the pairs of a row
      float2 x[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = quotient(v[i][2 * j], v[i][2 * j + 1]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (TRANSPOSE) {
          c[2 * j] = (e4m3x2(x[0][j].x, x[1][j].x) | (e4m3x2(x[2][j].x, x[3][j].x) << 16)) ^ kMinusCodes;
          c[2 * j + 1] = (e4m3x2(x[0][j].y, x[1][j].y) | (e4m3x2(x[2][j].y, x[3][j].y) << 16)) ^ kMinusCodes;
        } else {
          c[2 * j] = (e4m3x2(x[j][0].x, x[j][0].y) | (e4m3x2(x[j][1].x, x[j][1].y) << 16)) ^ kMinusCodes;
          c[2 * j + 1] = (e4m3x2(x[j][2].x, x[j][2].y) | (e4m3x2(x[j][3].x, x[j][3].y) << 16)) ^ kMinusCodes;
        }
      }
    };
    if (over.sure && finite)
      words([&](float x, float y) { return halves(over(pair_of(x, y))); });
    else
      words([&](float x, float y) { return make_float2(finite ? __fdiv_rn(-x, s) : -0.f, finite ? __fdiv_rn(-y, s) : -0.f); });
    if (TRANSPOSE) {
      uint8_t* out = codes + (e * K + k) * static_cast<int64_t>(N) + n;
#pragma unroll
      for (int j = 0; j < 8; ++j) *reinterpret_cast<uint32_t*>(out + j * static_cast<int64_t>(N)) = c[j];
    } else {
      uint8_t* out = codes + (e * N + n) * static_cast<int64_t>(K) + k;
#pragma unroll
      for (int i = 0; i < 4; ++i) *reinterpret_cast<uint2*>(out + i * static_cast<int64_t>(K)) = make_uint2(c[2 * i], c[2 * i + 1]);
    }
  }
}

// ------------------------------------------------------------------- launch

template <typename... Params, typename... Args>
cudaError_t launch_smem(void (*kernel)(Params...), dim3 grid, int threads, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), dim3 grid, int threads, cudaStream_t st, Args... args) {
  return launch_smem(kernel, grid, threads, 0, st, args...);
}

cudaError_t launch_backward(void (*kernel)(SwigluParams), size_t smem, dim3 grid, cudaStream_t st, const SwigluParams& p) {
  const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  return e == cudaSuccess ? launch_smem(kernel, grid, kThreads, smem, st, p) : e;
}

unsigned tiles_of(int64_t n) { return static_cast<unsigned>((n + kWide - 1) / kWide); }

// The format of a plain (mode FG_BF16) or 8-bit input, -1 for none.
int format_of(int mode, int type) {
  switch (mode) {
    case FG_BF16: return type == FG_TYPE_F32 ? kF32Rows : kBf16Rows;
    case FG_MXFP8_B32:
    case FG_MXFP4_FP8A: return kE8m0By32;
    case FG_MXFP8: return kE8m0By128;
    case FG_FP8_BLOCK128: return kF32By128;
    default: return -1;
  }
}

fg_status check_plain(const char* what, const char* name, const void* p, int64_t ld, int64_t cols, int type) {
  if (type != FG_TYPE_F32 && type != FG_TYPE_BF16) return fail(FG_ERR_INVALID_ARG, "%s: bad type %d", what, type);
  if (!p) return fail(FG_ERR_INVALID_ARG, "%s: null %s", what, name);
  if (ld < cols)
    return fail(FG_ERR_SHAPE, "%s: rows of %s are %lld apart, shorter than their %lld values", what, name, (long long)ld,
                (long long)cols);
  if (!aligned(p, 16) || ld * (type == FG_TYPE_F32 ? 4 : 2) % 16)
    return fail(FG_ERR_ALIGN, "%s: %s and its rows must be 16-byte aligned", what, name);
  return FG_OK;
}

fg_status check_8bit(const char* what, int mode, const void* codes, const void* scales) {
  if (!codes || !scales) return fail(FG_ERR_INVALID_ARG, "%s: null codes or scales", what);
  if (!aligned(codes, 16) || !aligned(scales, mode == FG_FP8_BLOCK128 ? 4 : 1))
    return fail(FG_ERR_ALIGN, "%s: codes must be 16-byte aligned, fp32 scales 4-byte", what);
  return FG_OK;
}

fg_status check_image(const char* what, const void* data, const void* sf, const void* desc) {
  if (!data || !sf || !desc) return fail(FG_ERR_INVALID_ARG, "%s: null image, scale image or descriptor", what);
  if (!aligned(data, 128) || !aligned(sf, 16)) return fail(FG_ERR_ALIGN, "%s: images must be 128-byte aligned, scale images 16-byte", what);
  return FG_OK;
}

}  // namespace

fg_status check_columns(const char* what, int64_t C, int64_t R, int E) {
  if (E < 1 || E > kMaxExperts) return fail(FG_ERR_SHAPE, "%s: E=%d outside 1..%d", what, E, kMaxExperts);
  if (C <= 0 || C % 128 || C > (int64_t(1) << 24))
    return fail(FG_ERR_SHAPE, "%s: %lld columns (a positive multiple of 128)", what, (long long)C);
  if (R < 0 || R > (int64_t(1) << 24) || column_slabs(R, E) * kPlaces > (int64_t(1) << 20))
    return fail(FG_ERR_SHAPE, "%s: R=%lld rows of %d experts need more than 2^20 places", what, (long long)R, E);
  return FG_OK;
}

}  // namespace fg

using namespace fg;

extern "C" {

fg_status fg_columns_size(int64_t C, int64_t R, int E, int64_t* places, uint64_t* data_bytes, uint64_t* sf_bytes) {
  if (!places || !data_bytes || !sf_bytes) return fail(FG_ERR_INVALID_ARG, "null output");
  fg_status s = check_columns("fg_columns_size", C, R, E);
  if (s != FG_OK) return s;
  *places = column_slabs(R, E) * kPlaces;
  *data_bytes = static_cast<uint64_t>(C) * *places;
  *sf_bytes = *data_bytes / 32;
  return FG_OK;
}

fg_status fg_quantize_columns(int mode, const void* x, const void* scales, int type, int64_t T, int64_t C, int64_t ldx,
                              const int32_t* rows, int64_t R, const int32_t* offsets, int E, void* data, void* sf,
                              fg_bshuf* desc_out, void* stream) {
  const char* what = "fg_quantize_columns";
  const int fmt = format_of(mode, type);
  if (fmt < 0) return fail(FG_ERR_INVALID_ARG, "%s: mode %d is neither bf16 (plain values) nor an 8-bit block format", what, mode);
  fg_status s = check_columns(what, C, R, E);
  if (s != FG_OK) return s;
  if (T < 0 || T > (int64_t(1) << 24)) return fail(FG_ERR_SHAPE, "%s: T=%lld", what, (long long)T);
  if (!rows && T < R) return fail(FG_ERR_SHAPE, "%s: x has %lld rows, fewer than R=%lld", what, (long long)T, (long long)R);
  if (R > 0 && T == 0) return fail(FG_ERR_SHAPE, "%s: no rows of x to gather from", what);
  if (R > 0) {
    if (mode == FG_BF16) {
      if (scales) return fail(FG_ERR_INVALID_ARG, "%s: plain values take no scales", what);
      if ((s = check_plain(what, "x", x, ldx, C, type)) != FG_OK) return s;
    } else {
      if ((s = check_8bit(what, mode, x, scales)) != FG_OK) return s;
      if (ldx != C) return fail(FG_ERR_SHAPE, "%s: rows of codes must be contiguous", what);
    }
  }
  if (!offsets && E != 1) return fail(FG_ERR_INVALID_ARG, "%s: null offsets with %d experts", what, E);
  if (!aligned(offsets, 4) || !aligned(rows, 4)) return fail(FG_ERR_ALIGN, "%s: offsets and rows must be 4-byte aligned", what);
  if ((s = check_image(what, data, sf, desc_out)) != FG_OK) return s;
  if ((s = check_arch()) != FG_OK) return s;
  const int64_t slabs = column_slabs(R, E);
  ColumnsParams p{{x, scales, ldx, C}, offsets, rows,
                  {static_cast<uint8_t*>(data), static_cast<uint8_t*>(sf), static_cast<int>(slabs)},
                  static_cast<int>(T), static_cast<int>(R), E};
  // column tiles are shared out over blocks until there are 32 for an SM (8: 129 us,
  // 16: 118, 32: 113, all: 118 for the rows below); slabs go in four parts where there
  // would be fewer blocks than the GPU holds
  const int64_t tiles = C / kWide, most = 4 * sm_count();
  const bool few = tiles * slabs < most;
  const dim3 grid(static_cast<unsigned>(few ? tiles : std::min(tiles, (32 * sm_count() + slabs - 1) / slabs)), static_cast<unsigned>(slabs),
                  few ? 4 : 1);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
  switch (fmt) {
    case kF32Rows: e = launch(columns_kernel<kF32Rows>, grid, kThreads, st, p); break;
    case kBf16Rows: e = launch(columns_kernel<kBf16Rows>, grid, kThreads, st, p); break;
    case kE8m0By32: e = launch(columns_kernel<kE8m0By32>, grid, kThreads, st, p); break;
    case kE8m0By128: e = launch(columns_kernel<kE8m0By128>, grid, kThreads, st, p); break;
    case kF32By128: e = launch(columns_kernel<kF32By128>, grid, kThreads, st, p); break;
  }
  if (e != cudaSuccess) return cuda_fail(e, "column quantiser's launch");
  column_descriptor(C, slabs * kPlaces, data, sf, desc_out);
  return FG_OK;
}

fg_status fg_swiglu_backward_workspace_size(int64_t R, int64_t K, int weighted, uint64_t* bytes) {
  if (!bytes) return fail(FG_ERR_INVALID_ARG, "null output");
  if (R < 0 || R > (int64_t(1) << 24) || K <= 0 || K > (int64_t(1) << 20))
    return fail(FG_ERR_SHAPE, "fg_swiglu_backward: R=%lld, K=%lld", (long long)R, (long long)K);
  *bytes = weighted ? static_cast<uint64_t>(R) * (K / 32) * 4 : 0;
  return FG_OK;
}

fg_status fg_swiglu_backward(int mode, const void* dy, int type, int64_t R, int64_t K, int64_t ldd, const void* saved,
                             const void* saved_scales, const float* weights, const int32_t* rows, const int32_t* slots,
                             int64_t T, int top_k, const int32_t* offsets, int E, void* codes, void* scales, void* dx,
                             float* dweights, void* dx_data, void* dx_sf, fg_bshuf* dx_desc, void* act_data, void* act_sf,
                             fg_bshuf* act_desc, void* workspace, uint64_t workspace_bytes, void* stream) {
  const char* what = "fg_swiglu_backward";
  const int fmt = mode == FG_BF16 ? -1 : format_of(mode, type);
  if (fmt < 0) return fail(FG_ERR_INVALID_ARG, "%s: mode %d keeps no 8-bit blocks", what, mode);
  if (type != FG_TYPE_F32 && type != FG_TYPE_BF16) return fail(FG_ERR_INVALID_ARG, "%s: bad type %d", what, type);
  const bool columns = dx_data || act_data, weighted = weights != nullptr;
  if (E < 1 || E > kMaxExperts) return fail(FG_ERR_SHAPE, "%s: E=%d outside 1..%d", what, E, kMaxExperts);
  if (!offsets && E != 1) return fail(FG_ERR_INVALID_ARG, "%s: null offsets with %d experts", what, E);
  uint64_t need = 0;
  fg_status s = fg_swiglu_backward_workspace_size(R, K, weighted, &need);
  if (s != FG_OK) return s;
  if (K % scale_block(fmt))
    return fail(FG_ERR_SHAPE, "%s: K=%lld must be a multiple of %d for %s", what, (long long)K, scale_block(fmt), mode_name(mode));
  if (columns) {
    if ((s = check_columns(what, K, R, E)) != FG_OK) return s;
    if ((s = check_image(what, dx_data, dx_sf, dx_desc)) != FG_OK) return s;
    if ((s = check_image(what, act_data, act_sf, act_desc)) != FG_OK) return s;
  }
  const int64_t slabs = column_slabs(R, E);
  if (slabs > 65535) return fail(FG_ERR_SHAPE, "%s: R=%lld too large", what, (long long)R);
  if (weighted) {
    if (!rows || !slots || !dweights) return fail(FG_ERR_INVALID_ARG, "%s: weights need rows, slots and dweights", what);
    if (top_k < 1 || top_k > kMaxTopK || T < 0 || T > (int64_t(1) << 24) || (R > 0 && T == 0))
      return fail(FG_ERR_SHAPE, "%s: T=%lld, top_k=%d (1..%d)", what, (long long)T, top_k, kMaxTopK);
    if (!aligned(weights, 4) || !aligned(rows, 4) || !aligned(slots, 4) || !aligned(dweights, 4))
      return fail(FG_ERR_ALIGN, "%s: a pointer is not aligned to its type", what);
    if (need && (!workspace || workspace_bytes < need))
      return fail(FG_ERR_WORKSPACE, "%s: needs a %llu-byte workspace", what, (unsigned long long)need);
    if (!aligned(workspace, 4)) return fail(FG_ERR_ALIGN, "%s: workspace must be 4-byte aligned", what);
  } else if (dweights) {
    return fail(FG_ERR_INVALID_ARG, "%s: dweights without weights", what);
  }
  if (R > 0) {
    if ((s = check_plain(what, "dy", dy, ldd, K, type)) != FG_OK) return s;
    if ((s = check_8bit(what, mode, saved, saved_scales)) != FG_OK) return s;
    if ((s = check_8bit(what, mode, codes, scales)) != FG_OK) return s;
    if (!aligned(dx, 16)) return fail(FG_ERR_ALIGN, "%s: dx must be 16-byte aligned", what);
  }
  if (!aligned(offsets, 4)) return fail(FG_ERR_ALIGN, "%s: offsets must be 4-byte aligned", what);
  if (R == 0 && !columns && !weighted) return FG_OK;
  if ((s = check_arch()) != FG_OK) return s;
  const Image none{nullptr, nullptr, 0};
  SwigluParams p{{dy, nullptr, ldd, K}, {saved, saved_scales, 2 * K, 2 * K}, weights, rows, slots, offsets,
                 static_cast<uint8_t*>(codes), scales, dx, weighted ? static_cast<float*>(workspace) : nullptr,
                 columns ? Image{static_cast<uint8_t*>(dx_data), static_cast<uint8_t*>(dx_sf), static_cast<int>(slabs)} : none,
                 columns ? Image{static_cast<uint8_t*>(act_data), static_cast<uint8_t*>(act_sf), static_cast<int>(slabs)} : none,
                 static_cast<int>(T), static_cast<int>(R), E, static_cast<int>(K), top_k, static_cast<int>(K / 32)};
  // column tiles are shared out over blocks until there are sixteen for an SM (12: 201
  // us, 24: 201, 32: 197 for the rows above)
  const int64_t tiles = tiles_of(K), shares = (16 * sm_count() + slabs - 1) / slabs;
  // (and slabs cut in four where there would be fewer blocks than the GPU holds)
  const bool few = tiles * slabs < 4 * static_cast<int64_t>(sm_count());
  const dim3 grid(static_cast<unsigned>(std::min(tiles, shares)), static_cast<unsigned>(slabs), few ? 4 : 1);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
#define FG_B(FMT_)                                                                                           \
  case FMT_:                                                                                                 \
    e = type == FG_TYPE_BF16 ? launch_backward(swiglu_backward_kernel<FMT_, __nv_bfloat16>,                  \
                                               2 * sizeof(Landing<__nv_bfloat16>), grid, st, p)              \
                             : launch_backward(swiglu_backward_kernel<FMT_, float>, 2 * sizeof(Landing<float>), grid, st, p); \
    break;
  switch (fmt) { FG_B(kE8m0By32) FG_B(kE8m0By128) FG_B(kF32By128) }
#undef FG_B
  if (e != cudaSuccess) return cuda_fail(e, "gated activation's backward launch");
  if (weighted && T > 0) {
    const int64_t choices = T * top_k;
    e = launch(dweights_kernel, dim3(static_cast<unsigned>((choices + 31) / 32)), 256, st, static_cast<const float*>(p.dots), slots,
               choices, p.R, p.dot_parts, dweights);
    if (e != cudaSuccess) return cuda_fail(e, "routing weights' gradient launch");
  }
  if (columns) {
    column_descriptor(2 * K, slabs * kPlaces, dx_data, dx_sf, dx_desc);
    column_descriptor(K, slabs * kPlaces, act_data, act_sf, act_desc);
  }
  return FG_OK;
}

fg_status fg_quantize_weight(int mode, const void* w, int type, int E, int64_t N, int64_t K, int64_t ldw, int64_t stride,
                             int transpose, void* codes, void* scales, void* stream) {
  const char* what = "fg_quantize_weight";
  if (mode != FG_FP8_BLOCK128)
    return fail(FG_ERR_INVALID_ARG, "%s: mode %d has no 128 x 128 blocks (fg_quantize does its rows)", what, mode);
  if (E < 1 || E > kMaxExperts) return fail(FG_ERR_SHAPE, "%s: E=%d outside 1..%d", what, E, kMaxExperts);
  if (N <= 0 || K <= 0 || N % 128 || K % 128 || N > (int64_t(1) << 20) || K > (int64_t(1) << 20))
    return fail(FG_ERR_SHAPE, "%s: N=%lld and K=%lld must be multiples of 128 up to 2^20", what, (long long)N, (long long)K);
  fg_status s = check_plain(what, "w", w, ldw, K, type);
  if (s != FG_OK) return s;
  if (E > 1 && (stride < 0 || stride * (type == FG_TYPE_F32 ? 4 : 2) % 16))
    return fail(FG_ERR_ALIGN, "%s: experts %lld elements apart (16-byte aligned, not negative)", what, (long long)stride);
  if ((s = check_8bit(what, mode, codes, scales)) != FG_OK) return s;
  if ((s = check_arch()) != FG_OK) return s;
  // two blocks of threads an SM, fp32's one by their shared memory
  const int64_t blocks = E * (N / 128) * (K / 128), most = (type == FG_TYPE_F32 ? 1 : 2) * static_cast<int64_t>(sm_count());
  if (blocks > INT32_MAX - most) return fail(FG_ERR_SHAPE, "%s: %d weights of %lld x %lld are too large", what, E, (long long)N, (long long)K);
  const dim3 grid(static_cast<unsigned>(std::min(blocks, most)));
  uint8_t* c = static_cast<uint8_t*>(codes);
  float* sc = static_cast<float*>(scales);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int n = static_cast<int>(N), k = static_cast<int>(K);
  auto run = [&](auto kernel, auto x) {
    const int smem = 2 * 4 * 16 * kWeightThreads * static_cast<int>(sizeof(*x) / 2);
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void*>(kernel), smem);
    return e == cudaSuccess ? launch_smem(kernel, grid, kWeightThreads, smem, st, x, ldw, stride, n, k, static_cast<int>(blocks), c, sc) : e;
  };
  cudaError_t e;
  if (type == FG_TYPE_BF16) {
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(w);
    e = transpose ? run(weight_kernel<__nv_bfloat16, true>, x) : run(weight_kernel<__nv_bfloat16, false>, x);
  } else {
    const float* x = static_cast<const float*>(w);
    e = transpose ? run(weight_kernel<float, true>, x) : run(weight_kernel<float, false>, x);
  }
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "weight quantiser's launch");
}

}  // extern "C"
