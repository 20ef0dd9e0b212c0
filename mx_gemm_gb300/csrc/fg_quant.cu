// Activations into the A operand's formats: quantisation of rows (plain, or
// of the gated activation silu(g) * u), and the residual addition with RMS
// norm whose output is quantised before it leaves the registers.
//
// Formats.  A row of K values is cut into blocks of 32 (MXFP8_B32, MXFP4,
// MXFP4_FP8A's activations) or 128 (MXFP8, FP8_BLOCK128).  For the MX formats
// the block's scale is the E8M0 code c = 127 + ceil(log2(amax / elem_max)),
// clamped to 0..254 (127 for an all-zero block), and a value's code is
// RNE(x * 2^(127 - c)) in the element format: 2^(c-127) is the smallest power
// of two that keeps the block inside the format.  FP8_BLOCK128 keeps the fp32
// scale amax / 448 (1 for an all-zero block; rounded up where amax < 2^-132),
// codes RNE(x / scale).  A block that holds a NaN or an infinity gets the NaN
// scale (E8M0 255, fp32 NaN) and zero codes, so whatever is computed from it is
// NaN.
//
// The ceil(log2()) needs no logarithm: amax = 1.m * 2^e and elem_max is 1.75 *
// 2^8 (e4m3) or 1.5 * 2^2 (e2m1), so it is e - 8 or e - 2, plus one where 1.m
// is above 1.75 or 1.5; exact on the bits, as is the product with a power of
// two.  The only rounding besides the code's own is that of the 32-bit value.
//
// Both kernels are bound by HBM: every input byte is read once (16 bytes a
// load) and every output byte written once.  Measured: 8191 x 7168 bf16 with
// residual to 32-K mxfp8 63.4 us (6.5 TB/s of the 6.8 that a copy reaches), the
// gated activation of 32761 x 2048 in 50 us (6.8 TB/s).  One row of 7168 takes 6.5
// us of host time, 4.6 us on the GPU, all latency: a block of 896 threads with
// one chunk each, the weight's load under way during the reduction.
#include <cuda_bf16.h>

#include "fg_host.cuh"
#include "fg_internal.cuh"
#include "fg_ptx.cuh"
#include "fg_values.cuh"

namespace fg {

namespace {

constexpr int kVec = 8;  // consecutive values per thread

// ------------------------------------------------------------ loads, codes

// Eight e2m1 codes, v[0] in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[kVec]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

constexpr int block_of(int mode) { return (mode == kMXFP8 || mode == kBlock) ? 128 : 32; }

// Quantise this thread's eight values of a block spread over block_of(MODE) / 8
// consecutive lanes and store codes and scale.  chunk: index of the eight
// values in the contiguous [M][K] output.  Every lane of the warp calls it;
// `live` lanes store.  BITS: the largest magnitude by whole numbers, two instructions a
// value, instead of half of one; it is the faster where the values come out of the
// fast power and reciprocal (the gated activation of 32761 x 2048 bf16: 48.8 us against
// 50.9) and the slower where they come from memory (32761 x 4096: 63.2 against 60.4), or
// with fp32 scales (the activation: 62.9 against 61.4).
template <int MODE, bool BITS = false>
__device__ __forceinline__ void quantize8(float (&v)[kVec], bool live, size_t chunk, void* codes, void* scales) {
  constexpr int LANES = block_of(MODE) / kVec;
  uint32_t amax = 0;  // of |v|'s bits: their order is that of the values, NaN above infinity
  if (BITS) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) amax = max(amax, __float_as_uint(v[i]) & 0x7fffffffu);
  } else {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < kVec; i += 2) most = largest(most, v[i], v[i + 1]);
    amax = __float_as_uint(most);
  }
#pragma unroll
  for (int d = 1; d < LANES; d *= 2) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
  const bool finite = amax < 0x7f800000u;
  const bool first = (threadIdx.x & (LANES - 1)) == 0;
  if (MODE == kBlock) {
    // v becomes the negative quotients.  The NaN scale is put in after them, which are
    // of zeros then.  (Divided by -s instead of negated, v takes six registers more, and
    // the norm of 8191 x 7168 a quarter of its warps: 72 us for 61.)
    const float s = f32_scale_of(finite ? amax : 0u);
    const Over over(s);
    if (over.sure && finite) {
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        const float2 q = halves(over(pair_of(v[i], v[i + 1])));
        v[i] = q.x;
        v[i + 1] = q.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = __fdiv_rn(finite ? -v[i] : -0.f, s);
    }
    if (live && first) static_cast<float*>(scales)[chunk / LANES] = finite ? s : __uint_as_float(0x7fc00000u);
  } else {
    constexpr int SHIFT = MODE == kMXFP4 ? 2 : 8;
    constexpr uint32_t TOP = MODE == kMXFP4 ? 0x400000u : 0x600000u;  // fraction bits of 1.5, 1.75: one more above them
    int c = static_cast<int>((amax + (0x7fffffu - TOP)) >> 23) - SHIFT;
    c = amax == 0 ? 127 : (c < 0 ? 0 : c);
    // a block of other than finite values: all codes zero
    const float f = __uint_as_float(static_cast<uint32_t>(254 - c) << 23);
#pragma unroll
    for (int i = 0; i < kVec; i += 2) mul2(v[i], v[i + 1], f, f);
    if (!finite) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = 0.f;
    }
    if (live && first) static_cast<uint8_t*>(scales)[chunk / LANES] = static_cast<uint8_t>(finite ? c : 255);
  }
  if (!live) return;
  if (MODE == kMXFP4) {
    static_cast<uint32_t*>(codes)[chunk] = e2m1x8(v);
  } else {
    constexpr uint32_t TURN = MODE == kBlock ? kMinusCodes : 0u;
    uint2 o;
    o.x = (e4m3x2(v[0], v[1]) | (e4m3x2(v[2], v[3]) << 16)) ^ TURN;
    o.y = (e4m3x2(v[4], v[5]) | (e4m3x2(v[6], v[7]) << 16)) ^ TURN;
    static_cast<uint2*>(codes)[chunk] = o;
  }
}

// --------------------------------------------------------------- quantise

// v = silu(v) * u = v / (1 + 2^(-v log2 e)) * u for two values, with the fast
// power and reciprocal (2 ulp each, and |v| 2^-24 from the rounded exponent,
// against the 2^-4 steps of the codes).  Zero below v = -88.7, where exp(-v) is
// past 32 bits.  Down to there 1 / (1 + exp(-v)) may be under 2^-126, which the
// fast reciprocal would flush: it takes a sixteenth of the sum.
__device__ __forceinline__ void swiglu2(float& v0, float& v1, float u0, float u1) {
  constexpr float kLog2e = 1.44269504088896341f;
  constexpr float kSixteenth = 0.0625f;
  float e0 = v0, e1 = v1;
  mul2(e0, e1, -kLog2e, -kLog2e);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e0));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e1));
  e0 = fmaf(e0, kSixteenth, kSixteenth);
  e1 = fmaf(e1, kSixteenth, kSixteenth);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e0));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e1));
  mul2(e0, e1, kSixteenth, kSixteenth);
  mul2(v0, v1, e0, e1);
  mul2(v0, v1, u0, u1);
}

// Threads (x, y) of a block take eight values of each of ROWS rows, blockDim.y
// apart: no division, and a warp's lanes never split a scale block.  With many
// rows a thread takes two: swiglu of 32761 x 2048 in 49.9 us (6.8 TB/s; 52.3 with
// four rows, 64.8 with eight, whose loads crowd out other blocks).
template <int MODE, int ACT, int ROWS, typename T>
__global__ void __launch_bounds__(256) quantize_kernel(const T* __restrict__ x, int64_t M, int64_t K, int64_t ldx,
                                                       void* __restrict__ codes, void* __restrict__ scales) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t cpr = K / kVec;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (blockDim.y * ROWS) + threadIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x;
  Raw8<T> a[ROWS], b[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t row = row0 + i * blockDim.y;
    a[i].zero();
    b[i].zero();
    if (row < M && c < cpr) {
      const T* src = x + row * ldx + c * kVec;
      a[i].load_once(src);
      if (ACT == FG_ACT_SWIGLU) b[i].load_once(src + K);
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t row = row0 + i * blockDim.y;
    float v[kVec];
    a[i].widen(v);
    if (ACT == FG_ACT_SWIGLU) {
      float u[kVec];
      b[i].widen(u);
#pragma unroll
      for (int j = 0; j < kVec; j += 2) swiglu2(v[j], v[j + 1], u[j], u[j + 1]);
    }
    quantize8<MODE, ACT == FG_ACT_SWIGLU && MODE != kBlock>(v, row < M && c < cpr, static_cast<size_t>(row * cpr + c), codes, scales);
  }
}

// The gated activation with its checkpoint: codes and scales of silu(g) * u, and
// of g and u themselves, as the forward pass of a training step keeps them.  One
// pass: 4 bytes read and 3 written per value of the activation, where three calls
// of the quantiser read 8.  Bound by HBM: 32761 x 2048 in 32-K blocks in 73.5 us
// (6.5 TB/s of the 6.8 that a copy reaches); in fp32 blocks of 128 in 110, whose scales'
// and quotients' instructions take longer.
template <int MODE, int ROWS, typename T>
__global__ void __launch_bounds__(256) checkpoint_kernel(const T* __restrict__ x, int64_t M, int64_t K, int64_t ldx,
                                                         void* __restrict__ codes, void* __restrict__ scales,
                                                         void* __restrict__ saved, void* __restrict__ saved_scales) {
  pdl_wait();
  pdl_launch_dependents();
  const int64_t cpr = K / kVec;
  const int64_t row0 = static_cast<int64_t>(blockIdx.x) * (blockDim.y * ROWS) + threadIdx.y;
  const int64_t c = static_cast<int64_t>(blockIdx.y) * blockDim.x + threadIdx.x;
  Raw8<T> a[ROWS], b[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t row = row0 + i * blockDim.y;
    a[i].zero();
    b[i].zero();
    if (row < M && c < cpr) {
      const T* src = x + row * ldx + c * kVec;
      a[i].load_once(src);
      b[i].load_once(src + K);
    }
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int64_t row = row0 + i * blockDim.y;
    const bool live = row < M && c < cpr;
    float v[kVec], g[kVec], u[kVec];
    a[i].widen(g);
    b[i].widen(u);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[j] = g[j];
#pragma unroll
    for (int j = 0; j < kVec; j += 2) swiglu2(v[j], v[j + 1], u[j], u[j + 1]);
    quantize8<MODE>(v, live, static_cast<size_t>(row * cpr + c), codes, scales);
    quantize8<MODE>(g, live, static_cast<size_t>(2 * row * cpr + c), saved, saved_scales);
    quantize8<MODE>(u, live, static_cast<size_t>((2 * row + 1) * cpr + c), saved, saved_scales);
  }
}

// -------------------------------------------------------- RMS norm, quantise

struct NormParams {
  const void* x;
  const void* residual;    // null: none
  const void* weight;
  void* residual_out;      // null: not wanted
  void* y;                 // null: not wanted
  void* codes;             // kBF16: null
  void* scales;
  int64_t ldx, ldr, K;
  float eps;
};

// One block per row; a thread keeps NC chunks of eight values in registers, so
// the row is read once.  MOST: threads of the block at most; with 1024 a thread
// has 64 registers and four chunks spill (8191 x 7168, 224 threads: 66.1 us so, 63.4
// with up to 128).
template <int MODE, typename T, int NC, int MOST>
__global__ void __launch_bounds__(MOST) rmsnorm_kernel(const NormParams p) {
  __shared__ float part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int cpr = static_cast<int>(p.K / kVec);
  const int64_t row = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(p.x) + row * p.ldx;
  const T* r = static_cast<const T*>(p.residual) + row * p.ldr;
  const T* w = static_cast<const T*>(p.weight);
  float v[NC][kVec];
  Raw8<T> g[NC];  // the weight, on its way during the reduction
  {
    Raw8<T> a[NC], b[NC];
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      a[i].zero();
      b[i].zero();
      g[i].zero();
      if (c < cpr) {
        a[i].load_once(x + c * kVec);
        if (p.residual) b[i].load_once(r + c * kVec);
      }
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < cpr) g[i].load(w + c * kVec);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      float u[kVec];
      a[i].widen(v[i]);
      b[i].widen(u);
      if (p.residual) {
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[i][j] += u[j];
      }
    }
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) ss = fmaf(v[i][j], v[i][j], ss);
  }
  if (p.residual_out) {
    T* out = static_cast<T*>(p.residual_out) + row * p.K;
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (c < cpr) store8(out + c * kVec, v[i]);
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if (lane == 0) part[warp] = ss;
  __syncthreads();
  ss = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d /= 2) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  const float inv = rsqrtf(ss / static_cast<float>(p.K) + p.eps);
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    const bool live = c < cpr;
    float u[kVec];
    g[i].widen(u);
#pragma unroll
    for (int j = 0; j < kVec; ++j) v[i][j] = v[i][j] * inv * u[j];
    if (live) {
      if (p.y) store8(static_cast<T*>(p.y) + row * p.K + c * kVec, v[i]);
    }
    if constexpr (MODE != kBF16)
      quantize8<MODE>(v[i], live, static_cast<size_t>(row) * cpr + c, p.codes, p.scales);
  }
}

// ------------------------------------------------------------------- launch

void pdl_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute& attr, dim3 grid, dim3 block, cudaStream_t st) {
  cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl_enabled() ? 1 : 0;
}

// Columns of threads for rows of cpr chunks: the widest of 16..256 that wastes no
// more of a row than the narrowest does.
int thread_columns(int64_t cpr) {
  int bx = 16;
  for (int b = 32; b <= 256; b *= 2)
    if ((cpr + b - 1) / b * b <= (cpr + 15) / 16 * 16) bx = b;
  return bx;
}

template <int MODE, typename T>
cudaError_t launch_checkpoint(const void* x, int64_t M, int64_t K, int64_t ldx, void* codes, void* scales, void* saved,
                              void* saved_scales, cudaStream_t st) {
  const int64_t cpr = K / kVec;
  const int bx = thread_columns(cpr), by = 256 / bx;
  const int64_t cols = (cpr + bx - 1) / bx;
  const bool many = (M + 2 * by - 1) / (2 * by) * cols >= 8 * sm_count();  // as in launch_quantize
  const int64_t rows = many ? 2 * by : by;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  pdl_config(cfg, attr, dim3(static_cast<unsigned>((M + rows - 1) / rows), static_cast<unsigned>(cols)), dim3(bx, by), st);
  const T* src = static_cast<const T*>(x);
  return many ? cudaLaunchKernelEx(&cfg, checkpoint_kernel<MODE, 2, T>, src, M, K, ldx, codes, scales, saved, saved_scales)
              : cudaLaunchKernelEx(&cfg, checkpoint_kernel<MODE, 1, T>, src, M, K, ldx, codes, scales, saved, saved_scales);
}

template <int MODE, int ACT, typename T>
cudaError_t launch_quantize(const void* x, int64_t M, int64_t K, int64_t ldx, void* codes, void* scales,
                            cudaStream_t st) {
  const int64_t cpr = K / kVec;
  const int bx = thread_columns(cpr), by = 256 / bx;
  const int64_t cols = (cpr + bx - 1) / bx;
  // two rows a thread once that leaves eight blocks for every SM
  const bool many = (M + 2 * by - 1) / (2 * by) * cols >= 8 * sm_count();
  const int64_t rows = many ? 2 * by : by;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  pdl_config(cfg, attr, dim3(static_cast<unsigned>((M + rows - 1) / rows), static_cast<unsigned>(cols)), dim3(bx, by), st);
  const T* src = static_cast<const T*>(x);
  return many ? cudaLaunchKernelEx(&cfg, quantize_kernel<MODE, ACT, 2, T>, src, M, K, ldx, codes, scales)
              : cudaLaunchKernelEx(&cfg, quantize_kernel<MODE, ACT, 1, T>, src, M, K, ldx, codes, scales);
}

template <int MODE, typename T>
cudaError_t launch_norm(const NormParams& p, int64_t M, cudaStream_t st) {
  const int64_t cpr = p.K / kVec;
  // four chunks a thread where there are rows enough to fill the GPU, one
  // (the shortest chain of loads) where there are not
  const int64_t want = M >= sm_count() ? 4 : 1;
  int nc = 1;
  while (nc < 4 && (nc < want || (cpr + nc - 1) / nc > 1024)) nc *= 2;
  int64_t threads = ((cpr + nc - 1) / nc + 31) / 32 * 32;
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr;
  pdl_config(cfg, attr, dim3(static_cast<unsigned>(M)), dim3(static_cast<unsigned>(threads)), st);
  switch (nc) {
    case 1: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<MODE, T, 1, 1024>, p);
    case 2: return cudaLaunchKernelEx(&cfg, rmsnorm_kernel<MODE, T, 2, 1024>, p);
    default:
      return threads <= 512 ? cudaLaunchKernelEx(&cfg, rmsnorm_kernel<MODE, T, 4, 512>, p)
                            : cudaLaunchKernelEx(&cfg, rmsnorm_kernel<MODE, T, 4, 1024>, p);
  }
}

fg_status check_rows(const char* what, int mode, int64_t M, int64_t K, int type) {
  if (type != FG_TYPE_F32 && type != FG_TYPE_BF16) return fail(FG_ERR_INVALID_ARG, "%s: bad type %d", what, type);
  if (M < 0 || K <= 0) return fail(FG_ERR_SHAPE, "%s: M=%lld, K=%lld", what, (long long)M, (long long)K);
  if (M > (int64_t(1) << 24) || K > (int64_t(1) << 20))
    return fail(FG_ERR_SHAPE, "%s: M=%lld or K=%lld too large", what, (long long)M, (long long)K);
  const int64_t blk = mode == FG_BF16 ? kVec : block_of(mode);
  if (K % blk)
    return fail(FG_ERR_SHAPE, "%s: K=%lld must be a multiple of %lld for %s", what, (long long)K, (long long)blk,
                mode_name(mode));
  return FG_OK;
}

// A row-major input whose rows are ld elements apart: whole 16-byte loads.
fg_status check_input(const char* what, const char* name, const void* p, int64_t ld, int64_t cols, int type) {
  if (!p) return fail(FG_ERR_INVALID_ARG, "%s: null %s", what, name);
  const int64_t es = type == FG_TYPE_F32 ? 4 : 2;
  if (ld < cols) return fail(FG_ERR_SHAPE, "%s: rows of %s are %lld apart, shorter than their %lld values", what, name,
                             (long long)ld, (long long)cols);
  if (!aligned(p, 16) || (ld * es) % 16)
    return fail(FG_ERR_ALIGN, "%s: %s and its rows must be 16-byte aligned", what, name);
  return FG_OK;
}

fg_status check_codes(const char* what, int mode, const void* codes, const void* scales) {
  if (!codes || !scales) return fail(FG_ERR_INVALID_ARG, "%s: null codes or scales", what);
  if (!aligned(codes, 16) || !aligned(scales, mode == FG_FP8_BLOCK128 ? 4 : 1))
    return fail(FG_ERR_ALIGN, "%s: codes must be 16-byte aligned, fp32 scales 4-byte", what);
  return FG_OK;
}

// The modes an activation is quantised for; the codes of MXFP4_FP8A's
// activations are those of MXFP8_B32.
bool quant_mode(int mode) { return mode == FG_FP8_BLOCK128 || is_mx(mode); }

}  // namespace

}  // namespace fg

using namespace fg;

extern "C" {

fg_status fg_quantize(int mode, int act, const void* x, int type, int64_t M, int64_t K, int64_t ldx, void* codes,
                      void* scales, void* stream) {
  if (!mode_ok(mode) || !quant_mode(mode))
    return fail(FG_ERR_INVALID_ARG, "fg_quantize: mode %d has no block scales to choose", mode);
  if (act != FG_ACT_NONE && act != FG_ACT_SWIGLU) return fail(FG_ERR_INVALID_ARG, "fg_quantize: bad act %d", act);
  fg_status s = check_rows("fg_quantize", mode, M, K, type);
  if (s != FG_OK) return s;
  if (M == 0) return FG_OK;
  if ((s = check_input("fg_quantize", "x", x, ldx, act == FG_ACT_SWIGLU ? 2 * K : K, type)) != FG_OK) return s;
  if ((s = check_codes("fg_quantize", mode, codes, scales)) != FG_OK) return s;
  if ((s = check_arch()) != FG_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
#define FG_Q(MODE_)                                                                                          \
  case MODE_:                                                                                                \
    if (type == FG_TYPE_BF16)                                                                                \
      e = act ? launch_quantize<MODE_, FG_ACT_SWIGLU, __nv_bfloat16>(x, M, K, ldx, codes, scales, st)        \
              : launch_quantize<MODE_, FG_ACT_NONE, __nv_bfloat16>(x, M, K, ldx, codes, scales, st);         \
    else                                                                                                     \
      e = act ? launch_quantize<MODE_, FG_ACT_SWIGLU, float>(x, M, K, ldx, codes, scales, st)                \
              : launch_quantize<MODE_, FG_ACT_NONE, float>(x, M, K, ldx, codes, scales, st);                 \
    break;
  switch (mode == FG_MXFP4_FP8A ? FG_MXFP8_B32 : mode) {
    FG_Q(FG_FP8_BLOCK128) FG_Q(FG_MXFP8) FG_Q(FG_MXFP4) FG_Q(FG_MXFP8_B32)
  }
#undef FG_Q
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "quantise launch");
}

fg_status fg_swiglu_checkpoint(int mode, const void* x, int type, int64_t M, int64_t K, int64_t ldx, void* codes,
                               void* scales, void* saved, void* saved_scales, void* stream) {
  const char* what = "fg_swiglu_checkpoint";
  if (!mode_ok(mode) || !quant_mode(mode) || mode == FG_MXFP4)
    return fail(FG_ERR_INVALID_ARG, "%s: mode %d keeps no 8-bit blocks", what, mode);
  fg_status s = check_rows(what, mode, M, K, type);
  if (s != FG_OK) return s;
  if (M == 0) return FG_OK;
  if ((s = check_input(what, "x", x, ldx, 2 * K, type)) != FG_OK) return s;
  if ((s = check_codes(what, mode, codes, scales)) != FG_OK) return s;
  if ((s = check_codes(what, mode, saved, saved_scales)) != FG_OK) return s;
  if ((s = check_arch()) != FG_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
#define FG_C(MODE_)                                                                                                      \
  case MODE_:                                                                                                            \
    e = type == FG_TYPE_BF16                                                                                             \
            ? launch_checkpoint<MODE_, __nv_bfloat16>(x, M, K, ldx, codes, scales, saved, saved_scales, st)              \
            : launch_checkpoint<MODE_, float>(x, M, K, ldx, codes, scales, saved, saved_scales, st);                     \
    break;
  switch (mode == FG_MXFP4_FP8A ? FG_MXFP8_B32 : mode) { FG_C(FG_FP8_BLOCK128) FG_C(FG_MXFP8) FG_C(FG_MXFP8_B32) }
#undef FG_C
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "checkpoint launch");
}

fg_status fg_rmsnorm_quantize(int mode, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                              const void* weight, float eps, int type, int64_t M, int64_t K, void* residual_out,
                              void* y, void* codes, void* scales, void* stream) {
  const char* what = "fg_rmsnorm_quantize";
  if (!mode_ok(mode) || (mode != FG_BF16 && !quant_mode(mode)))
    return fail(FG_ERR_INVALID_ARG, "%s: mode %d has no block scales to choose", what, mode);
  fg_status s = check_rows(what, mode, M, K, type);
  if (s != FG_OK) return s;
  if (K > 32768) return fail(FG_ERR_SHAPE, "%s: K=%lld above 32768 (a block keeps its row in registers)", what, (long long)K);
  if (!(eps >= 0.f)) return fail(FG_ERR_INVALID_ARG, "%s: eps must not be negative", what);
  if (M == 0) return FG_OK;
  if ((s = check_input(what, "x", x, ldx, K, type)) != FG_OK) return s;
  if (residual && (s = check_input(what, "residual", residual, ldr, K, type)) != FG_OK) return s;
  if ((s = check_input(what, "weight", weight, K, K, type)) != FG_OK) return s;
  if (mode == FG_BF16) {
    if (codes || scales) return fail(FG_ERR_INVALID_ARG, "%s: bf16 takes no codes or scales", what);
    if (!y) return fail(FG_ERR_INVALID_ARG, "%s: null y", what);
  } else if ((s = check_codes(what, mode, codes, scales)) != FG_OK) {
    return s;
  }
  if ((residual_out && !aligned(residual_out, 16)) || (y && !aligned(y, 16)))
    return fail(FG_ERR_ALIGN, "%s: outputs must be 16-byte aligned", what);
  if ((s = check_arch()) != FG_OK) return s;
  NormParams p{x, residual, weight, residual_out, y, codes, scales, ldx, ldr, K, eps};
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaErrorInvalidValue;
#define FG_N(MODE_)                                                     \
  case MODE_:                                                           \
    e = type == FG_TYPE_BF16 ? launch_norm<MODE_, __nv_bfloat16>(p, M, st) \
                             : launch_norm<MODE_, float>(p, M, st);     \
    break;
  switch (mode == FG_MXFP4_FP8A ? FG_MXFP8_B32 : mode) {
    FG_N(FG_BF16) FG_N(FG_FP8_BLOCK128) FG_N(FG_MXFP8) FG_N(FG_MXFP4) FG_N(FG_MXFP8_B32)
  }
#undef FG_N
  return e == cudaSuccess ? FG_OK : cuda_fail(e, "RMS norm launch");
}

}  // extern "C"
