// Rows of a recurrent state in registers, shared by the single-token steps:
// 8 columns a lane (16-byte accesses), K / 8 lanes a row.
#pragma once

#include "gdn_device.h"

namespace gdn {
namespace rows {

// Lane cl of LPR holds 8 columns of a state row: 8 cl .. 8 cl + 7 of a bf16
// pool (one 16-byte access); 4 cl .. + 3 and K / 2 + 4 cl .. + 3 of an fp32 one
// (two accesses that each cover a contiguous piece of the row).
template <typename S, int K> struct Cols;
template <int K> struct Cols<bf16_t, K> {
  static constexpr int second = 4;   // distance of the lane's columns 4 .. 7 from its first
  static __device__ __forceinline__ int first(int cl) { return 8 * cl; }
};
template <int K> struct Cols<float, K> {
  static constexpr int second = K / 2;
  static __device__ __forceinline__ int first(int cl) { return 4 * cl; }
};

__device__ __forceinline__ void unpack2(uint32_t w, float& a, float& b) {
  a = __builtin_bit_cast(float, w << 16);
  b = __builtin_bit_cast(float, w & 0xFFFF0000u);
}

// four consecutive values
__device__ __forceinline__ void load4(const bf16_t* p, float* f) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  unpack2(v.x, f[0], f[1]);
  unpack2(v.y, f[2], f[3]);
}
__device__ __forceinline__ void load4(const float* p, float* f) {
  const float4 v = *reinterpret_cast<const float4*>(p);
  f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
}

template <typename S> struct Raw;
template <> struct Raw<bf16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16_t* p, int) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    unpack2(v.x, f[0], f[1]);
    unpack2(v.y, f[2], f[3]);
    unpack2(v.z, f[4], f[5]);
    unpack2(v.w, f[6], f[7]);
  }
};
template <> struct Raw<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p, int second) {
    a = *reinterpret_cast<const f32x4*>(p);
    b = *reinterpret_cast<const f32x4*>(p + second);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a[e];
      f[4 + e] = b[e];
    }
  }
};
__device__ __forceinline__ void put_state(bf16_t* p, int, const float (&f)[8]) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  store_nt16(p, u4{pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7])});
}
__device__ __forceinline__ void put_state(float* p, int second, const float (&f)[8]) {
  store_nt16(p, f32x4{f[0], f[1], f[2], f[3]});
  store_nt16(p + second, f32x4{f[4], f[5], f[6], f[7]});
}

// Sum over the LPR lanes of a state row.
template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  x += dpp_f<0x141>(x);
  if constexpr (LPR == 16) x += dpp_f<0x140>(x);
  return x;
}

}  // namespace rows
}  // namespace gdn
