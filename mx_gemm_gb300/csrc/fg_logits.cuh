// Router logits of a token in a warp's registers: what routing, the balance loss
// and the logits' gradient share.
#pragma once
#include <cuda_bf16.h>

#include <cstdint>

namespace fg {

// exp(l - top), 1 where both are infinite
__device__ __forceinline__ float exp_below(float l, float top) { return l == top ? 1.f : expf(l - top); }

// A lane's logits of one token: chunks of V consecutive experts, 32 chunks (one
// a lane) next to one another.
template <typename T, int VPL>
struct Logits {
  static constexpr int V = VPL * sizeof(T) < 16 ? VPL : 16 / sizeof(T);
  uint32_t bits[VPL];

  static __device__ __forceinline__ int expert(int i, int lane) { return ((i / V) * 32 + lane) * V + i % V; }

  // p: logits, ldl (elements from token to token), E, whole (rows aligned to a chunk)
  template <typename P>
  __device__ __forceinline__ void load(const P& p, int64_t t, int lane) {
    const T* row = static_cast<const T*>(p.logits) + t * p.ldl;
    constexpr uint32_t NONE = sizeof(T) == 2 ? 0xff80u : 0xff800000u;  // -infinity
#pragma unroll
    for (int c = 0; c < VPL; c += V) {
      const int e = expert(c, lane);
      constexpr int BYTES = V * sizeof(T);
      uint32_t w[(BYTES + 3) / 4];
      if (p.whole && e + V <= p.E) {
        if constexpr (BYTES == 16) {
          const uint4 u = __ldcs(reinterpret_cast<const uint4*>(row + e));
          w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
        } else if constexpr (BYTES == 8) {
          const uint2 u = __ldcs(reinterpret_cast<const uint2*>(row + e));
          w[0] = u.x; w[1] = u.y;
        } else if constexpr (BYTES == 4) {
          w[0] = __ldcs(reinterpret_cast<const uint32_t*>(row + e));
        } else {
          w[0] = __ldcs(reinterpret_cast<const unsigned short*>(row + e));
        }
#pragma unroll
        for (int i = 0; i < V; ++i)
          bits[c + i] = sizeof(T) == 4 ? w[i] : ((w[i / 2] >> (16 * (i % 2))) & 0xffffu);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          bits[c + i] = NONE;
          if (e + i < p.E)
            bits[c + i] = sizeof(T) == 4 ? __ldcs(reinterpret_cast<const uint32_t*>(row) + e + i)
                                         : __ldcs(reinterpret_cast<const unsigned short*>(row) + e + i);
        }
      }
    }
  }
};

}  // namespace fg
