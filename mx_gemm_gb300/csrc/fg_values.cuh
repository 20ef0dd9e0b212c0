// Values on their way between memory and registers, eight at a time, and the
// scales and codes of 8-bit blocks: what the kernels of fg_quant.cu and
// fg_columns.cu share.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace fg {

// Eight values as they lie in memory: loads are issued together and widened
// when they are used.  once: not read again, so kept out of the caches' way.
template <typename T>
struct Raw8 {
  uint4 q[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) q[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void load_once(const T* p) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) q[i] = __ldcs(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) q[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void widen(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i) {
      const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (sizeof(T) == 2) {
          v[2 * j] = __uint_as_float(w[j] << 16);
          v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          v[4 * i + j] = __uint_as_float(w[j]);
        }
      }
    }
  }
};

__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// a0 *= b0, a1 *= b1 in one instruction, each rounded once.
__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%0, %1};\n mov.b64 b, {%2, %3};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}

// Two 32-bit values in neighbouring registers, and arithmetic on both at once, each
// rounded once.  Kept as pairs from load to store they need no moves.
using Pair = unsigned long long;
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
  Pair p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}
__device__ __forceinline__ float2 halves(Pair p) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(p));
  return f;
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  Pair p;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair p;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(p) : "l"(a), "l"(b));
  return p;
}
__device__ __forceinline__ Pair fma(Pair a, Pair b, Pair c) {
  Pair p;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(p) : "l"(a), "l"(b), "l"(c));
  return p;
}

// The largest of three magnitudes; NaN if one is.
__device__ __forceinline__ float largest(float a, float b, float c) {
  float m;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
  return m;
}

// Two codes, `lo` in the lower half.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// E8M0 code of a block of e4m3 values whose largest magnitude has these bits:
// 127 + ceil(log2(amax / 448)), at least 0, 127 for zero (not for infinities and NaN).
__device__ __forceinline__ int e8m0_of(uint32_t amax) {
  const int c = max(static_cast<int>((amax + 0x1fffffu) >> 23) - 8, 0);  // one more where the fraction is above 1.75's
  return amax == 0 ? 127 : c;
}

// 2^(127 - c), what values are multiplied by, and 2^(c - 127), what codes stand for
// (NaN for 255).
__device__ __forceinline__ float e8m0_down(int c) { return __uint_as_float(static_cast<uint32_t>(254 - c) << 23); }
__device__ __forceinline__ float e8m0_up(uint32_t c) {
  return __uint_as_float(c == 0u ? 0x400000u : (c == 255u ? 0x7fc00000u : c << 23));
}

// fp32 scale of a block of e4m3 values: amax / 448 (1 for zero); below 2^-132,
// where the quotient has nine bits at most, rounded up on the bits as multiples
// of 2^-149, so that no code saturates and nothing is divided by zero.
__device__ __forceinline__ float f32_scale_of(uint32_t amax) {
  return amax == 0 ? 1.f
                   : (amax < (1u << 17) ? __uint_as_float((amax + 447u) / 448u) : __fdiv_rn(__uint_as_float(amax), 448.f));
}

// -(v / s) for a block's fp32 scale s, rounded to nearest: with r = 1 / s rounded to nearest
// and q = v r, the remainder v - q s is exact in one fused multiply-add and q + (v - q s)
// r is the quotient (Markstein 1990, "Computation of elementary functions on the IBM RISC
// System/6000 processor").  Three instructions for two values, where a division takes ten
// for one (a checkpoint of 32761 x 2048: 154 us with divisions, 109 so).  It holds while the
// remainder is a multiple of fp32's smallest step, 2^-149: with q >= 2^a and s >= 2^b it is
// one of 2^(a + b - 46).  Quotients below half an e4m3 step, 2^-10, have code 0 whatever
// their last bits, so b >= -93 is enough; `sure` keeps three powers of two from there, and
// r and all products from the ends of fp32.
//
// Every sign is turned: of v = -0 this leaves +0, where q + (v - q s) r, a sum of zeros of
// both signs, would be +0 for either.  The codes' sign bits are turned back (kMinusCodes).
struct Over {
  Pair minus_r, s2;
  bool sure;
  __device__ __forceinline__ explicit Over(float s) {
    const float x = -__frcp_rn(s);
    minus_r = pair_of(x, x);
    s2 = pair_of(s, s);
    sure = s >= 0x1p-90f && s < 0x1p100f;
  }
  __device__ __forceinline__ Pair operator()(Pair v) const {
    const Pair q = mul(v, minus_r);
    return fma(fma(q, s2, v), minus_r, q);
  }
};
constexpr uint32_t kMinusCodes = 0x80808080u;  // sign bits of four codes

// Two values of two e4m3 codes, the lower half's first.
__device__ __forceinline__ float2 e4m3_values(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

}  // namespace fg
