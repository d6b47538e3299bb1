// Delta-rule step with one gate per key channel, T = 1 .. 4 tokens over a pool
// of states, gfx950.  Per batch row and v-head, token by token,
//
//   e_c = exp(-exp(A_log) softplus(a_c + dt_bias_c))      (key channel c)
//   d   = beta (v - S (e o k)),  o = S (e o q) + (k . q) d
//   S  <- S diag(e) + d k^T
//
// with beta = sigmoid(b), k over its L2 norm, q over its norm times the scale:
// the recurrence of the per-channel-gated prefill, whose decayed state's two
// products are taken from the state before the decay, so that both row sums of
// a token run together, in front of its update.
//
// HBM-bound by the state, which moves twice (2 x 32 KiB per head at K = V = 128 in
// bf16), as long as the vector work stays below that: 4 K V operations a token, with
// four tokens about as long as the transfer.  So what a token's rows have in common
// (gates, normalised q and k, k . q, beta) is computed once a work-group and read from
// LDS, and outputs are added up in a way that leaves each to one lane.  256 rows x 32
// heads of four tokens: 123 us, 580 MB at 4.7 TB/s (150 us with q and k in every wave,
// registers for three waves a SIMD and outputs summed in all lanes; a large copy reaches
// 5.2 TB/s); one token a row: 108 us, 5.1 TB/s, 512 rows 213 us; an fp32 pool, 256 rows:
// 215 us with one token (5.0 TB/s), 209 with four.  One row of 32 heads, one token: 4.6 us,
// the launch and two trips to memory.
//
// A work-group of V K / 64 threads takes one (row, head), also when these are fewer than
// the CUs (32 of them, one token: 4.1 us a launch in a graph; four times as many
// work-groups of a wave each: 4.9, and 155 instead of 115 us for the 8192 of above).
// K / 8 lanes of a DPP row hold whole state rows: row sums are in-row reductions.  The
// state's loads are issued before everything else.  States and sums are fp32; the
// pool's type rounds once, at the end.

#include "gdn_device.h"
#include "mixer_launch.h"
#include "ssm_rate.h"
#include "state_rows.h"

namespace gdn {

namespace {

using namespace rows;

// by value: a choice between two elements of an array would be one between addresses
__device__ __forceinline__ float choose(bool c, float x, float y) { return c ? x : y; }

// x[cl % 8]
__device__ __forceinline__ float pick(const float (&x)[8], int cl) {
  const bool b0 = cl & 1, b1 = cl & 2, b2 = cl & 4;
  const float lo = choose(b1, choose(b0, x[3], x[2]), choose(b0, x[1], x[0]));
  const float hi = choose(b1, choose(b0, x[7], x[6]), choose(b0, x[5], x[4]));
  return choose(b2, hi, lo);
}

// Sums over the LPR lanes of a state row of the eight values x; lane cl gets that of
// x[cl % 8].  Halves of the lanes swap halves of the values: 8 additions instead of
// the 24 (32) of eight sums that every lane gets.
template <int LPR>
__device__ __forceinline__ float row_sum_each(const float (&x)[8], int cl) {
  const bool b0 = cl & 1, b1 = cl & 2, b2 = cl & 4;
  float y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) y[i] = choose(b2, x[4 + i], x[i]) + dpp_f<0x141>(choose(b2, x[i], x[4 + i]));
  const float p = choose(b1, y[2], y[0]) + dpp_f<0x4E>(choose(b1, y[0], y[2]));
  const float q = choose(b1, y[3], y[1]) + dpp_f<0x4E>(choose(b1, y[1], y[3]));
  float r = choose(b0, q, p) + dpp_f<0xB1>(choose(b0, p, q));
  if constexpr (LPR == 16) r += dpp_f<0x128>(r);   // the lane 8 further on
  return r;
}

// sqrt(sum of x^2 + eps) of a row of LPR lanes.  Squares that leave fp32's range or
// its normal numbers: x becomes x times a power of two, and the result is of that.
template <int LPR>
__device__ __forceinline__ float row_norm(float (&x)[8], float eps) {
  float s = 0.f;
#pragma unroll
  for (int c = 0; c < 8; ++c) s = fmaf(x[c], x[c], s);
  s = row_sum<LPR>(s) + eps;
  if (!(s >= 0x1p-100f && s <= 0x1p100f)) {
    const float f = s < 1.f ? 0x1p100f : 0x1p-80f;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      x[c] *= f;
      s = fmaf(x[c], x[c], s);
    }
    s = row_sum<LPR>(s) + eps * f * f;
  }
  return sqrtf(s);
}

// exp(A_log) step for A_log > FAST_RATE: step is softplus(bu) / beta where `soft`, which
// underflows where the product may not (there it is e^bu / beta).
__device__ __forceinline__ double fast_rate(float A_log, float bu, bool soft, float step, float beta) {
  if (soft && bu < -20.f) return (double)expf((float)((double)A_log + (double)bu)) / (double)beta;
  return rate_of(A_log) * (double)step;
}

// T: io type, S: pool type.  A thread holds R = 8 consecutive state rows.
template <typename T, typename S, int K, int V, int TT>
__global__ __launch_bounds__(V * K / 64) __attribute__((amdgpu_waves_per_eu(4))) void kda_decode_kernel(KdaStepArgs a) {
  constexpr int LPR = K / 8, R = 8, TPB = V * K / 64;
  __shared__ __attribute__((aligned(16))) float gate[TT][K];
  __shared__ __attribute__((aligned(16))) float kn[TT][K];
  __shared__ __attribute__((aligned(16))) float qn[TT][K];
  __shared__ __attribute__((aligned(16))) float vs[TT][V];
  __shared__ float scal[TT][2];   // k . q, beta
  const int bi = blockIdx.x / a.HV;
  const int hv = blockIdx.x - bi * a.HV;
  const int hk = hv / (a.HV / a.H);
  const int cl = threadIdx.x % LPR;
  const int row0 = threadIdx.x / LPR * R;
  const int slot = a.idx ? a.idx[bi] : bi;
  const bool valid = slot >= 0 && slot < a.pool;
  T* const op = reinterpret_cast<T*>(a.o) + ((size_t)bi * TT * a.HV + hv) * V + row0;
  if (!valid) {   // o = 0, the pool is not touched (the whole work-group leaves)
    if (cl < R) {
#pragma unroll
      for (int t = 0; t < TT; ++t) op[(size_t)t * a.HV * V + cl] = from_f<T>(0.f);
    }
    return;
  }
  constexpr int second = Cols<S, K>::second;
  const int c0 = Cols<S, K>::first(cl);
  S* sp = reinterpret_cast<S*>(a.state) + (((size_t)slot * a.HV + hv) * V + row0) * K + c0;
  Raw<S> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i].load(sp + (size_t)i * K, second);

  const size_t tok0 = (size_t)bi * TT;
  const T* ap = reinterpret_cast<const T*>(a.a) + (tok0 * a.HV + hv) * K;
  const T* vp = reinterpret_cast<const T*>(a.v) + (tok0 * a.HV + hv) * V;
  for (int i = threadIdx.x; i < TT * V / 4; i += TPB) {
    const int t = i / (V / 4), r = i % (V / 4) * 4;
    load4(vp + (size_t)t * a.HV * V + r, &vs[t][r]);
  }
  const float A_log = a.A_log[hv];
  const float A = -expf(A_log);
  const bool fast = A_log > FAST_RATE;   // uniform
  for (int i = threadIdx.x; i < TT * K; i += TPB) {
    const int t = i / K, c = i % K;
    const float u = to_f(ap[(size_t)t * a.HV * K + c]) + a.dt_bias[(size_t)hv * K + c];
    const float bu = a.sp_beta * u;
    const float step = bu <= a.sp_thr ? log1pf(expf(bu)) / a.sp_beta : u;
    float Ad = A * step;
    if (fast) Ad = -(float)fast_rate(A_log, bu, bu <= a.sp_thr, step, a.sp_beta);
    gate[t][c] = expf(Ad);
  }
  // q, k and the scalars of a token: LPR lanes of the last wave each
  if (const int t = ((int)threadIdx.x - (TPB - 64)) / LPR; (int)threadIdx.x >= TPB - 64 && t < TT) {
    const size_t at = ((tok0 + t) * a.H + hk) * K + c0;
    const T* qp = reinterpret_cast<const T*>(a.q) + at;
    const T* kp = reinterpret_cast<const T*>(a.k) + at;
    float q[8], k[8];
    load4(qp, q);
    load4(qp + second, q + 4);
    load4(kp, k);
    load4(kp + second, k + 4);
    const float bt = to_f(reinterpret_cast<const T*>(a.b)[(tok0 + t) * a.HV + hv]);
    float qs = a.scale, ks = 1.f;
    if (a.use_norm) {
      qs = a.scale / row_norm<LPR>(q, a.eps);
      ks = 1.f / row_norm<LPR>(k, a.eps);
    }
    float kq = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) kq = fmaf(k[c], q[c], kq);
    kq = row_sum<LPR>(kq);
    float* const kw = &kn[t][c0];
    float* const qw = &qn[t][c0];
    *reinterpret_cast<f32x4*>(kw) = f32x4{k[0], k[1], k[2], k[3]} * ks;
    *reinterpret_cast<f32x4*>(kw + second) = f32x4{k[4], k[5], k[6], k[7]} * ks;
    *reinterpret_cast<f32x4*>(qw) = f32x4{q[0], q[1], q[2], q[3]} * qs;
    *reinterpret_cast<f32x4*>(qw + second) = f32x4{q[4], q[5], q[6], q[7]} * qs;
    if (cl == 0) {
      scal[t][0] = kq * (qs * ks);
      scal[t][1] = 1.f / (1.f + expf(-bt));
    }
  }
  __syncthreads();

  float st[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i].get(st[i]);

#pragma unroll 1
  for (int t = 0; t < TT; ++t) {
    float e[8], ek[8], eq[8], k[8], v[R];
    load4(&vs[t][row0], v);
    load4(&vs[t][row0 + 4], v + 4);
    load4(&gate[t][c0], e);
    load4(&gate[t][c0 + second], e + 4);
    load4(&kn[t][c0], k);
    load4(&kn[t][c0 + second], k + 4);
    load4(&qn[t][c0], eq);
    load4(&qn[t][c0 + second], eq + 4);
    const float kq = scal[t][0], bt = scal[t][1];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ek[c] = e[c] * k[c];
      eq[c] *= e[c];
    }
    float dlt[R], out[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float p = 0.f, o = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        p = fmaf(st[i][c], ek[c], p);
        o = fmaf(st[i][c], eq[c], o);
      }
      dlt[i] = p;
      out[i] = o;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      dlt[i] = bt * (v[i] - row_sum<LPR>(dlt[i]));
#pragma unroll
      for (int c = 0; c < 8; ++c) st[i][c] = fmaf(dlt[i], k[c], st[i][c] * e[c]);
    }
    // lane i of the row group stores row i
    const float y = fmaf(kq, pick(dlt, cl), row_sum_each<LPR>(out, cl));
    if (cl < R) op[(size_t)t * a.HV * V + cl] = from_f<T>(y);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) put_state(sp + (size_t)i * K, second, st[i]);
}

template <typename T, typename S, int K, int V>
hipError_t launch_v(const KdaStepArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((long long)a.B * a.HV)), threads(V * K / 64);
  switch (a.T) {
    case 1: hipLaunchKernelGGL((kda_decode_kernel<T, S, K, V, 1>), grid, threads, 0, s, a); break;
    case 2: hipLaunchKernelGGL((kda_decode_kernel<T, S, K, V, 2>), grid, threads, 0, s, a); break;
    case 3: hipLaunchKernelGGL((kda_decode_kernel<T, S, K, V, 3>), grid, threads, 0, s, a); break;
    default: hipLaunchKernelGGL((kda_decode_kernel<T, S, K, V, 4>), grid, threads, 0, s, a);
  }
  return hipGetLastError();
}

template <typename T, typename S, int K>
hipError_t launch_k(const KdaStepArgs& a, hipStream_t s) {
  return a.V == 128 ? launch_v<T, S, K, 128>(a, s) : launch_v<T, S, K, 64>(a, s);
}

template <typename T>
hipError_t launch_io(const KdaStepArgs& a, hipStream_t s) {
  if (a.state_bf16) return a.K == 128 ? launch_k<T, bf16_t, 128>(a, s) : launch_k<T, bf16_t, 64>(a, s);
  return a.K == 128 ? launch_k<T, float, 128>(a, s) : launch_k<T, float, 64>(a, s);
}

}  // namespace

hipError_t launch_kda_decode(const KdaStepArgs& a, hipStream_t s) {
  return a.bf16 ? launch_io<bf16_t>(a, s) : launch_io<float>(a, s);
}

}  // namespace gdn
