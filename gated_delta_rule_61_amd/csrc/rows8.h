// Eight consecutive channels of a token's row a lane (16 bytes of bf16), and
// what the row kernels of the convolution and the norm share around them.
#pragma once

#include "gdn_device.h"

namespace gdn {
namespace rows8 {

// 8 consecutive channels in memory
template <typename T> struct Raw8;
template <> struct Raw8<bf16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __builtin_bit_cast(float, w[e] << 16);
      f[2 * e + 1] = __builtin_bit_cast(float, w[e] & 0xFFFF0000u);
    }
  }
};
template <> struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void put8(bf16_t* p, const float (&f)[8]) {
  *reinterpret_cast<u32x4*>(p) =
      u32x4{pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7])};
}
__device__ __forceinline__ void put8(float* p, const float (&f)[8]) {
  *reinterpret_cast<f32x4*>(p) = f32x4{f[0], f[1], f[2], f[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{f[4], f[5], f[6], f[7]};
}

// ... as streaming stores
__device__ __forceinline__ void put8_nt(bf16_t* p, const float (&f)[8]) {
  store_nt16(p, u32x4{pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7])});
}
__device__ __forceinline__ void put8_nt(float* p, const float (&f)[8]) {
  store_nt16(p, f32x4{f[0], f[1], f[2], f[3]});
  store_nt16(p + 4, f32x4{f[4], f[5], f[6], f[7]});
}

__device__ __forceinline__ float silu_f(float a) {
  return a * __builtin_amdgcn_rcpf(1.0f + __expf(-a));
}

// Sum over the LPH lanes that hold one head (8 or 16 lanes of a DPP row).
template <int LPH>
__device__ __forceinline__ float head_sum(float x) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  x += dpp_f<0x141>(x);
  if constexpr (LPH == 16) x += dpp_f<0x140>(x);
  return x;
}

// First sequence whose boundary is at or behind `t` (N if none): a 64-way
// search, one load per level, the same result in every lane.
__device__ __forceinline__ int first_seq_from(const int64_t* cu, int N, long long t, int lane) {
  int lo = 0, hi = N;
  while (lo < hi) {
    const int step = (hi - lo + 63) / 64;
    const int i = lo + lane * step;
    const bool before = i < hi && (long long)cu[i] < t;
    const int cnt = __popcll(__ballot(before));
    if (step == 1) return lo + cnt;
    if (cnt == 0) return lo;
    const int top = lo + cnt * step;
    lo += (cnt - 1) * step + 1;
    hi = hi < top ? hi : top;
  }
  return lo;
}

}  // namespace rows8
}  // namespace gdn
