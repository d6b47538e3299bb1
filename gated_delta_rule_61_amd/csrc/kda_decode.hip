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
// HBM-bound: the state moves twice (2 x 32 KiB per head at K = V = 128 in
// bf16).  A work-group of 256 threads takes one (row, head), or four of 64
// threads a quarter of its value rows each when there are too few for the chip.
// K / 8 lanes of a DPP row hold whole state rows: row sums are in-row
// reductions.  The gates are the only thing threads share: each of the K T
// exponentials is computed once a work-group and read from LDS.  The state's
// loads are issued before everything else.

#include "gdn_device.h"
#include "mixer_launch.h"
#include "state_rows.h"

namespace gdn {

namespace {

using namespace rows;

// T: io type, S: pool type.  A thread holds R = 8 consecutive state rows.
template <typename T, typename S, int K, int TT, int TPB>
__global__ __launch_bounds__(TPB) void kda_decode_kernel(KdaStepArgs a, int parts) {
  constexpr int LPR = K / 8, R = 8;
  __shared__ __attribute__((aligned(16))) float gate[TT][K];
  const int bh = blockIdx.x / parts;
  const int part = blockIdx.x - bh * parts;
  const int bi = bh / a.HV;
  const int hv = bh - bi * a.HV;
  const int hk = hv / (a.HV / a.H);
  const int cl = threadIdx.x % LPR;
  const int row0 = (part * (TPB / LPR) + threadIdx.x / LPR) * R;   // < V: the launch has V K / 64 threads a state
  const int slot = a.idx ? a.idx[bi] : bi;
  const bool valid = slot >= 0 && slot < a.pool;
  T* const op = reinterpret_cast<T*>(a.o) + ((size_t)bi * TT * a.HV + hv) * a.V + row0;
  if (!valid) {   // o = 0, the pool is not touched (the whole work-group leaves)
    if (cl < R) {
#pragma unroll
      for (int t = 0; t < TT; ++t) op[(size_t)t * a.HV * a.V + cl] = from_f<T>(0.f);
    }
    return;
  }
  constexpr int second = Cols<S, K>::second;
  const int c0 = Cols<S, K>::first(cl);
  S* sp = reinterpret_cast<S*>(a.state) + (((size_t)slot * a.HV + hv) * a.V + row0) * K + c0;
  Raw<S> raw[R];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i].load(sp + (size_t)i * K, second);

  const size_t tok0 = (size_t)bi * TT;
  const T* ap = reinterpret_cast<const T*>(a.a) + (tok0 * a.HV + hv) * K;
  const T* qp = reinterpret_cast<const T*>(a.q) + (tok0 * a.H + hk) * K + c0;
  const T* kp = reinterpret_cast<const T*>(a.k) + (tok0 * a.H + hk) * K + c0;
  const T* vp = reinterpret_cast<const T*>(a.v) + (tok0 * a.HV + hv) * a.V + row0;
  float qq[TT][8], kk[TT][8], vv[TT][R], beta[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    load4(qp + (size_t)t * a.H * K, qq[t]);
    load4(qp + (size_t)t * a.H * K + second, qq[t] + 4);
    load4(kp + (size_t)t * a.H * K, kk[t]);
    load4(kp + (size_t)t * a.H * K + second, kk[t] + 4);
    load4(vp + (size_t)t * a.HV * a.V, vv[t]);
    load4(vp + (size_t)t * a.HV * a.V + 4, vv[t] + 4);
    beta[t] = to_f(reinterpret_cast<const T*>(a.b)[(tok0 + t) * a.HV + hv]);
  }
  const float A = -expf(a.A_log[hv]);
  for (int i = threadIdx.x; i < TT * K; i += TPB) {
    const int t = i / K, c = i % K;
    const float u = to_f(ap[(size_t)t * a.HV * K + c]) + a.dt_bias[(size_t)hv * K + c];
    const float bu = a.sp_beta * u;
    const float step = bu <= a.sp_thr ? log1pf(expf(bu)) / a.sp_beta : u;
    gate[t][c] = step == 0.f ? 1.f : expf(A * step);   // A may be infinite
  }
  __syncthreads();

  float st[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i) raw[i].get(st[i]);

#pragma unroll
  for (int t = 0; t < TT; ++t) {
    float e[8];
    load4(&gate[t][c0], e);
    load4(&gate[t][c0 + second], e + 4);
    float sq = 0.f, sk = 0.f, kq = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      sq = fmaf(qq[t][c], qq[t][c], sq);
      sk = fmaf(kk[t][c], kk[t][c], sk);
      kq = fmaf(kk[t][c], qq[t][c], kq);
    }
    kq = row_sum<LPR>(kq);
    float qs = a.scale, ks = 1.f;
    if (a.use_norm) {
      qs = a.scale / sqrtf(row_sum<LPR>(sq) + a.eps);
      ks = 1.f / sqrtf(row_sum<LPR>(sk) + a.eps);
    }
    kq *= qs * ks;
    float ek[8], eq[8], kn[8];
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      kn[c] = kk[t][c] * ks;
      ek[c] = e[c] * kn[c];
      eq[c] = e[c] * (qq[t][c] * qs);
    }
    const float bt = 1.f / (1.f + expf(-beta[t]));
    float pred[R], out[R];
#pragma unroll
    for (int i = 0; i < R; ++i) {
      float p = 0.f, o = 0.f;
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        p = fmaf(st[i][c], ek[c], p);
        o = fmaf(st[i][c], eq[c], o);
      }
      pred[i] = p;
      out[i] = o;
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      pred[i] = row_sum<LPR>(pred[i]);
      out[i] = row_sum<LPR>(out[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float dlt = bt * (vv[t][i] - pred[i]);
      out[i] = fmaf(kq, dlt, out[i]);
#pragma unroll
      for (int c = 0; c < 8; ++c) st[i][c] = fmaf(dlt, kn[c], st[i][c] * e[c]);
    }
    // lane i of the row group stores row i
    float y = out[0];
#pragma unroll
    for (int i = 1; i < R; ++i) y = cl == i ? out[i] : y;
    if (cl < R) op[(size_t)t * a.HV * a.V + cl] = from_f<T>(y);
  }
#pragma unroll
  for (int i = 0; i < R; ++i) put_state(sp + (size_t)i * K, second, st[i]);
}

template <typename T, typename S, int K, int TT>
hipError_t launch_t(const KdaStepArgs& a, hipStream_t s) {
  const long long pairs = (long long)a.B * a.HV;
  const int threads = a.V * (K / 8) / 8;   // 64, 128 or 256 threads hold a state
  // fewer (row, head) pairs than CUs, or a small state: work-groups of one wave
  if constexpr (K == 128) {
    if (pairs >= 256 && threads == 256) {
      hipLaunchKernelGGL((kda_decode_kernel<T, S, K, TT, 256>), dim3((unsigned)pairs), dim3(256), 0, s, a, 1);
      return hipGetLastError();
    }
  }
  const int parts = threads / 64;
  hipLaunchKernelGGL((kda_decode_kernel<T, S, K, TT, 64>), dim3((unsigned)(pairs * parts)), dim3(64), 0, s, a, parts);
  return hipGetLastError();
}

template <typename T, typename S, int K>
hipError_t launch_k(const KdaStepArgs& a, hipStream_t s) {
  switch (a.T) {
    case 1: return launch_t<T, S, K, 1>(a, s);
    case 2: return launch_t<T, S, K, 2>(a, s);
    case 3: return launch_t<T, S, K, 3>(a, s);
    default: return launch_t<T, S, K, 4>(a, s);
  }
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
