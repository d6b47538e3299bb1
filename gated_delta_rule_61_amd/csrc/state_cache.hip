// 8-bit cache of recurrent states, gfx950: states of fp32 (a prefill's ht,
// fp32 snapshots) or bf16 (a decode pool, bf16 snapshots) are quantised as they
// are written into cache slots, one scale per state row, and read back into
// fp32 (an initial state) or bf16 (a decode pool).
//
//   int8:  s = max(max|row| r, 2^-126), r = 1/127 rounded to fp32; code = the
//          exact quotient row / s rounded to nearest, ties to even
//   e4m3:  s = the smallest power of two >= 2^-126 with max|row| / s <= 448, so
//          that row / s is exact and the one rounding is the code's own (a
//          power of two costs a floating-point code at most one bit of its
//          17.8 binades of range and no precision)
//   read:  code * s, rounded once to the target's type
//
// A row with an infinity or NaN gets the scale NaN and codes 0, and so reads
// back as NaN throughout: a broken state is not turned into a plausible one.
//
// Memory-bound: 5 bytes per element with fp32 states (3 with bf16), ~10 VALU
// operations.  8 elements of a row per lane (two 16-byte accesses of fp32, 8
// bytes of codes), K / 8 lanes a row, the row's maximum by 3 or 4 in-row DPP
// steps; large stores take two rows a lane, whose loads are issued before the first
// maximum.
//
// Measured, states of 32 heads of 128 x 128: 128 fp32 ones stored as e4m3 60 us, 5.6
// TB/s (int8 64 us; a large copy 5.1 TB/s); 256 read back into bf16 78 us, 5.2 TB/s;
// one stored 3 us, one read 2.5.

#include "gdn_device.h"
#include "mixer_launch.h"

namespace gdn {

namespace {

template <typename T> struct Wide8;
template <> struct Wide8<bf16_t> {
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
template <> struct Wide8<float> {
  f32x4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p));
    b = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + 4));
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = a[e];
      f[4 + e] = b[e];
    }
  }
};

template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t x) {
  const uint32_t y = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xF, 0xF, false);
  return x > y ? x : y;
}

// x / s to the nearest integer, ties to even, exactly: the rounded product with
// the reciprocal is at most one off, and its remainder x - q s is exact in fp32
// (|q| < 128 and |x - q s| <= s: a multiple of the smaller of the last places of
// x and s that fits 24 bits).
__device__ __forceinline__ int quotient_even(float x, float s, float inv) {
  float q = rintf(x * inv);
  const float r = fmaf(-q, s, x), h = 0.5f * s, m = fabsf(r);
  if (m > h || (m == h && ((int)q & 1))) q += r > 0.f ? 1.0f : -1.0f;
  return (int)q;
}

struct Place {
  long long wide, code;   // element offset of the state's row in the wide array; row of the cache
  bool ok;
};

template <bool STORE>
__device__ __forceinline__ Place place(const StateQ8Args& a, long long row, long long rows, long long per) {
  Place p{0, 0, false};
  if (row >= rows) return p;
  const int n = (int)(row / per);
  const long long in = row - (long long)n * per;
  const int src = a.src_idx ? a.src_idx[n] : n, dst = a.dst_idx ? a.dst_idx[n] : n;
  const int w = STORE ? src : dst, q = STORE ? dst : src;
  if (w < 0 || w >= a.wide_n || q < 0 || q >= a.pool) return p;
  p.wide = ((long long)w * per + in) * a.K;
  p.code = (long long)q * per + in;
  p.ok = true;
  return p;
}

// ROWS: rows of a lane
template <typename T, int K, bool E4M3, int ROWS>
__global__ __launch_bounds__(256) void state_store_q8_kernel(StateQ8Args a, long long rows, long long per) {
  constexpr int LPR = K / 8, RPB = 256 / LPR;
  const int cl = threadIdx.x % LPR;
  const long long row0 = (long long)blockIdx.x * (RPB * ROWS) + threadIdx.x / LPR;
  Place p[ROWS];
  Wide8<T> raw[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    p[i] = place<true>(a, row0 + i * RPB, rows, per);
    if (p[i].ok) raw[i].load(reinterpret_cast<const T*>(a.wide) + p[i].wide + 8 * cl);
  }
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    if (!p[i].ok) continue;   // uniform over the lanes of a row
    float f[8];
    raw[i].get(f);
    uint32_t m = 0;   // bits of max|row|: a NaN is above infinity, which is above every number
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t b = __builtin_bit_cast(uint32_t, f[e]) & 0x7FFFFFFFu;
      m = m > b ? m : b;
    }
    m = dpp_max<0xB1>(m);
    m = dpp_max<0x4E>(m);
    m = dpp_max<0x141>(m);
    if constexpr (LPR == 16) m = dpp_max<0x140>(m);
    const bool bad = m >= 0x7F800000u;
    float scale;
    uint2 w;
    if constexpr (E4M3) {
      // max = 1.f 2^(E - 127): the scale's exponent is E - 8, one more where 1.f > 1.75
      int e = (int)(m >> 23) - 8 + ((m & 0x7FFFFFu) > 0x600000u ? 1 : 0);
      e = e < 1 ? 1 : e;
      scale = __builtin_bit_cast(float, (uint32_t)e << 23);
      const float inv = bad ? 0.f : __builtin_bit_cast(float, (uint32_t)(254 - e) << 23);
#pragma unroll
      for (int e2 = 0; e2 < 8; ++e2) f[e2] = bad ? 0.f : f[e2] * inv;
      int lo = 0, hi = 0;
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[0], f[1], lo, false);
      lo = __builtin_amdgcn_cvt_pk_fp8_f32(f[2], f[3], lo, true);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[4], f[5], hi, false);
      hi = __builtin_amdgcn_cvt_pk_fp8_f32(f[6], f[7], hi, true);
      w = uint2{(uint32_t)lo, (uint32_t)hi};
    } else {
      const float s = __builtin_bit_cast(float, m) * (1.0f / 127.0f);
      scale = s > 0x1p-126f ? s : 0x1p-126f;
      const float inv = 1.0f / scale;
      uint32_t c[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = bad ? 0u : (uint32_t)quotient_even(f[e], scale, inv) & 0xFFu;
      w = uint2{c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24, c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24};
    }
    if (bad) scale = __builtin_nanf("");
    store_nt8(reinterpret_cast<uint8_t*>(a.q8) + p[i].code * K + 8 * cl, w);
    if (cl == 0) a.scales[p[i].code] = scale;
  }
}

// One row a lane: with nothing between a load and its store, more waves hide the
// latency better than two rows do (256 states into bf16 78 us, two rows 85).
template <typename T, int K, bool E4M3>
__global__ __launch_bounds__(256) void state_load_q8_kernel(StateQ8Args a, long long rows, long long per) {
  constexpr int LPR = K / 8, RPB = 256 / LPR;
  const int cl = threadIdx.x % LPR;
  typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
  const Place p = place<false>(a, (long long)blockIdx.x * RPB + threadIdx.x / LPR, rows, per);
  if (!p.ok) return;
  const u32x2 raw = __builtin_nontemporal_load(
      reinterpret_cast<const u32x2*>(reinterpret_cast<const uint8_t*>(a.q8) + p.code * K + 8 * cl));
  const float scale = a.scales[p.code];
  float f[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (E4M3) {
      const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[h], false);
      const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[h], true);
      f[4 * h] = lo[0]; f[4 * h + 1] = lo[1]; f[4 * h + 2] = hi[0]; f[4 * h + 3] = hi[1];
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) f[4 * h + e] = (float)(int8_t)(raw[h] >> (8 * e));
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] *= scale;
  T* dst = reinterpret_cast<T*>(a.wide) + p.wide + 8 * cl;
  if constexpr (sizeof(T) == 2) {
    typedef uint32_t u4 __attribute__((ext_vector_type(4)));
    store_nt16(dst, u4{pack_bf2(f[0], f[1]), pack_bf2(f[2], f[3]), pack_bf2(f[4], f[5]), pack_bf2(f[6], f[7])});
  } else {
    store_nt16(dst, f32x4{f[0], f[1], f[2], f[3]});
    store_nt16(dst + 4, f32x4{f[4], f[5], f[6], f[7]});
  }
}

template <bool STORE, typename T, int K, bool E4M3>
hipError_t launch(const StateQ8Args& a, hipStream_t s) {
  const long long per = (long long)a.HV * a.V, rows = per * a.N;
  // Stores of fewer than 2^17 rows take one row a lane (states of 4096 rows of 128
  // fp32 as int8, one / two rows: 1 state 3.0 / 4.1 us, 16 10.6 / 10.7, 32
  // 19.4 / 19.2, 128 66 / 64).
  const int per_lane = STORE && rows >= (1 << 17) ? 2 : 1;
  const int per_block = 256 / (K / 8) * per_lane;
  const dim3 grid((unsigned)((rows + per_block - 1) / per_block)), block(256);
  if constexpr (STORE) {
    if (per_lane == 2) hipLaunchKernelGGL((state_store_q8_kernel<T, K, E4M3, 2>), grid, block, 0, s, a, rows, per);
    else hipLaunchKernelGGL((state_store_q8_kernel<T, K, E4M3, 1>), grid, block, 0, s, a, rows, per);
  } else {
    hipLaunchKernelGGL((state_load_q8_kernel<T, K, E4M3>), grid, block, 0, s, a, rows, per);
  }
  return hipGetLastError();
}

template <bool STORE>
hipError_t dispatch(const StateQ8Args& a, hipStream_t s) {
  if (a.wide_bf16) {
    if (a.K == 128) return a.e4m3 ? launch<STORE, bf16_t, 128, true>(a, s) : launch<STORE, bf16_t, 128, false>(a, s);
    return a.e4m3 ? launch<STORE, bf16_t, 64, true>(a, s) : launch<STORE, bf16_t, 64, false>(a, s);
  }
  if (a.K == 128) return a.e4m3 ? launch<STORE, float, 128, true>(a, s) : launch<STORE, float, 128, false>(a, s);
  return a.e4m3 ? launch<STORE, float, 64, true>(a, s) : launch<STORE, float, 64, false>(a, s);
}

}  // namespace

hipError_t launch_state_store_q8(const StateQ8Args& a, hipStream_t s) { return dispatch<true>(a, s); }
hipError_t launch_state_load_q8(const StateQ8Args& a, hipStream_t s) { return dispatch<false>(a, s); }

}  // namespace gdn
