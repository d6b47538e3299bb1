// Selective state-space step for T = 1 .. 4 tokens over a pool of states,
// gfx950.  Per batch row and head, token by token,
//
//   D_t = softplus(dt_t + dt_bias),  a_t = exp(-exp(A_log) D_t)
//   S  <- a_t S + (D_t x_t) B_t^T,   y_t = (S C_t + D x_t) silu(z_t)
//
// with S [V, K] read from the row's slot once, carried in fp32 across the
// tokens and written back once (fp32, or rounded to nearest-even bf16).
//
// HBM-bound: the state moves twice (2 x 64 KiB per head at V = K = 128 in
// fp32) against 5 operations an element and token.  Work-groups of 256 threads
// take one (row, head), or four work-groups of 64 threads a quarter of its
// value rows each when there are too few for the chip (rows are independent).
// K / 8 lanes of a DPP row hold whole state rows: the C product is a 3- or
// 4-step in-row reduction, without LDS or barriers, and every state access is
// 16 bytes a lane.  The state's loads are issued before everything else.
//
// Measured, 32 heads of 128 x 128: 256 rows over an fp32 pool 1.08 GB in 214 us,
// 5.1 TB/s (a large copy's rate); over a bf16 pool 112 us, 4.9 TB/s; one row 3.6 us.

#include "gdn_device.h"
#include "mixer_launch.h"
#include "ssm_rate.h"
#include "state_rows.h"

namespace gdn {

namespace {

using namespace rows;

// T: io type, S: pool type.  A thread holds R = 8 consecutive state rows.
template <typename T, typename S, int K, int TT, int TPB>
__global__ __launch_bounds__(TPB) void ssm_step_kernel(SsmArgs a, int parts) {
  constexpr int LPR = K / 8, R = 8;
  const int bh = blockIdx.x / parts;
  const int part = blockIdx.x - bh * parts;
  const int bi = bh / a.HV;
  const int hv = bh - bi * a.HV;
  const int hk = hv / (a.HV / a.Hk);
  const int cl = threadIdx.x % LPR;
  const int row0 = (part * (TPB / LPR) + threadIdx.x / LPR) * R;
  if (row0 >= a.V) return;
  const int slot = a.idx ? a.idx[bi] : bi;
  const bool valid = slot >= 0 && slot < a.pool;
  constexpr int second = Cols<S, K>::second;
  const int c0 = Cols<S, K>::first(cl);
  S* sp = reinterpret_cast<S*>(a.state) + (((size_t)(valid ? slot : 0) * a.HV + hv) * a.V + row0) * K + c0;
  Raw<S> raw[R];
  if (valid) {
#pragma unroll
    for (int i = 0; i < R; ++i) raw[i].load(sp + (size_t)i * K, second);
  }
  const T* xp = reinterpret_cast<const T*>(a.x.p) + (long long)bi * a.x.batch + (long long)hv * a.V + row0;
  const T* zp = reinterpret_cast<const T*>(a.z.p) + (long long)bi * a.z.batch + (long long)hv * a.V + row0;
  const T* dp = reinterpret_cast<const T*>(a.dt.p) + (long long)bi * a.dt.batch + hv;
  const T* bp = reinterpret_cast<const T*>(a.B.p) + (long long)bi * a.B.batch + (long long)hk * K + c0;
  const T* cp = reinterpret_cast<const T*>(a.C.p) + (long long)bi * a.C.batch + (long long)hk * K + c0;
  T* yp = reinterpret_cast<T*>(a.y) + ((long long)bi * TT * a.HV + hv) * a.V + row0;

  if (!valid) {   // y = 0, the pool is not touched
    if (cl < R) {
#pragma unroll
      for (int t = 0; t < TT; ++t) yp[(long long)t * a.HV * a.V + cl] = from_f<T>(0.f);
    }
    return;
  }

  float bb[TT][8], cc[TT][8], xx[TT][R], dt[TT], zz[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    load4(bp + t * a.B.token, bb[t]);
    load4(bp + t * a.B.token + second, bb[t] + 4);
    load4(cp + t * a.C.token, cc[t]);
    load4(cp + t * a.C.token + second, cc[t] + 4);
    load4(xp + t * a.x.token, xx[t]);
    load4(xp + t * a.x.token + 4, xx[t] + 4);
    dt[t] = to_f(dp[t * a.dt.token]);
    zz[t] = a.z.p ? to_f(zp[t * a.z.token + (cl & 7)]) : 0.f;
  }
  const float A_log = a.A_log[hv];
  const float A = -expf(A_log);
  const bool fast = A_log > FAST_RATE;
  const float bias = a.dt_bias ? a.dt_bias[hv] : 0.f;
  const float skip = a.D ? a.D[hv] : 0.f;

  float st[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i].get(st[i]);

#pragma unroll
  for (int t = 0; t < TT; ++t) {
    const float u = dt[t] + bias;
    float d = u;
    if (a.softplus) d = u <= 20.f ? log1pf(expf(u)) : u;
    float Ad = A * d;
    if (fast) Ad = -(float)(a.softplus ? fast_decay(A_log, u) : rate_of(A_log) * (double)d);
    const float alpha = expf(Ad);
    float out[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float dx = d * xx[t][i];
      float acc = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        st[i][e] = fmaf(dx, bb[t][e], alpha * st[i][e]);
        acc = fmaf(st[i][e], cc[t][e], acc);
      }
      out[i] = acc;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) out[i] = row_sum<LPR>(out[i]);
    // lane i of the row group finishes row i
    float y = out[0], xi = xx[t][0];
#pragma unroll
    for (int i = 1; i < R; ++i) {
      y = cl == i ? out[i] : y;
      xi = cl == i ? xx[t][i] : xi;
    }
    y = fmaf(skip, xi, y);
    if (a.z.p) y *= zz[t] * __builtin_amdgcn_rcpf(1.0f + __expf(-zz[t]));
    if (cl < R) yp[(long long)t * a.HV * a.V + cl] = from_f<T>(y);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) put_state(sp + (size_t)i * K, second, st[i]);
}

template <typename T, typename S, int K, int TT>
hipError_t launch_t(const SsmArgs& a, hipStream_t s) {
  const long long pairs = (long long)a.nb * a.HV;
  const int threads = a.V * (K / 8) / 8;   // 64, 128 or 256 threads hold a state
  // fewer (row, head) pairs than CUs, or a small state: work-groups of one wave
  // (fp32 pool, 32 heads of 128 x 128, one wave / four: 1 row 3.6 / 4.3 us, 4 rows
  // 5.0 / 5.3, 8 rows 7.5 / 7.0, 256 rows 216 / 214)
  if (pairs < 256 || threads < 256) {
    const int parts = threads / 64;
    hipLaunchKernelGGL((ssm_step_kernel<T, S, K, TT, 64>), dim3((unsigned)(pairs * parts)), dim3(64), 0, s, a, parts);
  } else {
    hipLaunchKernelGGL((ssm_step_kernel<T, S, K, TT, 256>), dim3((unsigned)pairs), dim3(256), 0, s, a, 1);
  }
  return hipGetLastError();
}

template <typename T, typename S, int K>
hipError_t launch_k(const SsmArgs& a, hipStream_t s) {
  switch (a.T) {
    case 1: return launch_t<T, S, K, 1>(a, s);
    case 2: return launch_t<T, S, K, 2>(a, s);
    case 3: return launch_t<T, S, K, 3>(a, s);
    default: return launch_t<T, S, K, 4>(a, s);
  }
}

template <typename T>
hipError_t launch_io(const SsmArgs& a, hipStream_t s) {
  if (a.state_bf16) return a.K == 128 ? launch_k<T, bf16_t, 128>(a, s) : launch_k<T, bf16_t, 64>(a, s);
  return a.K == 128 ? launch_k<T, float, 128>(a, s) : launch_k<T, float, 64>(a, s);
}

}  // namespace

hipError_t launch_ssm_step(const SsmArgs& a, hipStream_t s) {
  return a.bf16 ? launch_io<bf16_t>(a, s) : launch_io<float>(a, s);
}

}  // namespace gdn
