// Gradients of the short causal depthwise convolution, gfx950.  With
//
//   c_t = bias + sum_{j < W} w_j x_{t - W + 1 + j},  u = silu(c) (or c),
//   y = u, or every head of the leading sections over sqrt(sum u^2 + eps)
//
// and dy the gradient of y:
//
//   du = dy, or r (dy - n (n . dy)) with n = r u, r = 1 / sqrt(sum u^2 + eps)
//   dc = du silu'(c)
//   dx_t = sum_j w_j dc_{t + W - 1 - j}    (rows of the same sequence)
//   dw_j = sum_t dc_t x_{t - W + 1 + j},   dbias = sum_t dc_t
//
// Three rows of D channels (x, dy, dx) against 6 W + ~20 operations a value, which take
// about as long as the transfer: 16001 packed tokens of 8192 bf16 channels with head
// norms 172 us, 826 MB at 4.8 TB/s (a large copy reaches 5.2; the vector units are busy
// seven tenths of it, with the two waves a SIMD that 215 registers leave); 4096 fp32
// channels: 168 us, 4.7 TB/s, with head norms or without.  c is computed again from x,
// nothing is kept from the forward pass.  As there, a lane owns 8 consecutive channels
// and walks down a run of tokens: the last W - 1 rows of x and the W open sums of dx stay
// in registers, and so do the sums of dw and dbias.  The W - 1 rows of dc behind a run
// are computed a second time for the run's last dx.
// Blocks of rows that are all the run's own go without checks of its end (180 -> 172
// us; loading them a block ahead gave nothing more).  All sums are fp32.  Each run
// leaves one row of sums in a workspace; a second launch adds them up in a fixed order
// (6 us).

#include <type_traits>

#include "gdn_device.h"
#include "mixer_launch.h"
#include "rows8.h"

namespace gdn {

namespace {

using namespace rows8;

// NORM: lanes of a head, or 0.  A wave handles 512 channels of `run` tokens.
template <typename T, int W, int NORM>
__global__ __launch_bounds__(64) void conv_bwd_kernel(ConvBwdArgs a, int run, int cblocks) {
  constexpr int U = 4;   // rows loaded together
  const int lane = threadIdx.x;
  const int r = blockIdx.x / cblocks;
  const int c = ((blockIdx.x - r * cblocks) * 64 + lane) * 8;
  const bool live = c < a.D;
  const int cc = live ? c : 0;
  const long long total = (long long)a.B * a.T;
  const long long t0 = (long long)r * run;
  const long long t1 = t0 + run < total ? t0 + run : total;

  float w[W][8], bias[8] = {}, dw[W][8] = {}, db[8] = {};
  {
    const T* wp = reinterpret_cast<const T*>(a.weight) + (size_t)cc * W;
    float flat[8 * W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      Raw8<T> raw;
      raw.load(wp + 8 * i);
      float f[8];
      raw.get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) flat[8 * i + e] = f[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
    if (a.bias) {
      Raw8<T> raw;
      raw.load(reinterpret_cast<const T*>(a.bias) + cc);
      raw.get(bias);
    }
  }
  const int sec = (cc >= a.end[0]) + (cc >= a.end[1]);
  const int lo = sec == 0 ? 0 : (sec == 1 ? a.end[0] : a.end[1]);
  const int hi = sec == 0 ? a.end[0] : (sec == 1 ? a.end[1] : a.end[2]);
  const T* const gb = reinterpret_cast<const T*>(sec == 0 ? a.dout[0] : (sec == 1 ? a.dout[1] : a.dout[2])) + (cc - lo);
  const long long gw = hi - lo;
  const bool norm = sec < a.norm_sections;
  const T* const xb = reinterpret_cast<const T*>(a.x.p) + cc;
  T* const dxb = reinterpret_cast<T*>(a.dx) + cc;

  auto bound = [&](int n) -> long long {   // clamped boundary n
    if (!a.cu) return (long long)n * a.T;
    const long long v = (long long)a.cu[n];
    return v < 0 ? 0 : (v > total ? total : v);
  };
  // the sequence that holds t0
  int s;
  if (a.cu) {
    s = __builtin_amdgcn_readfirstlane(first_seq_from(a.cu, a.N, t0 + 1, lane)) - 1;
    s = s < 0 ? 0 : s;
  } else {
    s = (int)(t0 / a.T);
  }
  for (; s < a.N; ++s) {
    const long long start = bound(s), end = bound(s + 1);
    if (start >= t1) break;
    const long long from = start > t0 ? start : t0;
    const long long own = end < t1 ? end : t1;    // dx, dw and dbias of [from, own)
    if (from >= own) continue;
    const long long stop = own + W - 1 < end ? own + W - 1 : end;
    auto x_row = [&](long long t) -> const T* {
      return a.cu ? xb + t * a.x.token : xb + (long long)s * a.x.batch + (t - start) * a.x.token;
    };
    float win[W - 1][8];   // the last W - 1 rows of x
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const long long t = from - (W - 1) + j;
      Raw8<T> raw = {};
      if (t >= start) raw.load(x_row(t));
      raw.get(win[j]);
    }
    float open[W][8] = {};   // sums of dx_{t-W+1} .. dx_t
    // rows t .. t + U - 1; WHOLE: all of them this run's own
    auto rows = [&](long long t, auto whole) __attribute__((always_inline)) {
      constexpr bool WHOLE = decltype(whole)::value;
      Raw8<T> xr[U], gr[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long tt = WHOLE || t + u < stop ? t + u : stop - 1;
        xr[u].load(x_row(tt));
        gr[u].load(gb + tt * gw);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (!WHOLE && t + u >= stop) break;
        float x[8], g[8], y[8];
        xr[u].get(x);
        gr[u].get(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float acc = bias[e];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) acc = fmaf(w[j][e], win[j][e], acc);
          y[e] = fmaf(w[W - 1][e], x[e], acc);
        }
        float slope[8];
        if (a.silu) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float p = __builtin_amdgcn_rcpf(1.0f + __expf(-y[e]));
            y[e] *= p;
            slope[e] = fmaf(y[e], 1.0f - p, p);   // y may be large: 1 - p is 0 there, p + y would round p away
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) slope[e] = 1.0f;
        }
        if constexpr (NORM != 0) {
          float q = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) q = fmaf(y[e], y[e], q);
          q = head_sum<NORM>(q) + a.eps;
          float k = 1.0f;
          // squares that leave fp32's range or its normal numbers: once more from the
          // head times a power of two, eps times its square
          if (norm && !(q >= 0x1p-100f && q <= 0x1p100f)) {
            k = q < 1.0f ? 0x1p100f : 0x1p-70f;
            q = 0.f;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              y[e] *= k;
              q = fmaf(y[e], y[e], q);
            }
            q = head_sum<NORM>(q) + a.eps * k * k;
          }
          const float rs = __builtin_amdgcn_rsqf(q);
          float dot = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            y[e] *= rs;
            dot = fmaf(y[e], g[e], dot);
          }
          dot = head_sum<NORM>(dot);
          if (norm) {
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = rs * k * (g[e] - y[e] * dot);
          }
        }
        const bool mine = WHOLE || t + u < own;   // uniform
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float dc = g[e] * slope[e];
#pragma unroll
          for (int j = 0; j < W; ++j) open[j][e] = fmaf(w[j][e], dc, open[j][e]);
          if (mine) {
#pragma unroll
            for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(dc, win[j][e], dw[j][e]);
            dw[W - 1][e] = fmaf(dc, x[e], dw[W - 1][e]);
            db[e] += dc;
          }
        }
        // dx_{t-W+1} is whole; it belongs to this run from `from` on
        if (t + u - (W - 1) >= from && live) put8(dxb + (t + u - (W - 1)) * a.D, open[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
#pragma unroll
          for (int j = 0; j + 1 < W; ++j) open[j][e] = open[j + 1][e];
          open[W - 1][e] = 0.f;
#pragma unroll
          for (int j = 0; j + 2 < W; ++j) win[j][e] = win[j + 1][e];
          win[W - 2][e] = x[e];
        }
      }
    };
    long long t = from;
    for (; t + U <= own; t += U) rows(t, std::true_type{});
    for (; t < stop; t += U) rows(t, std::false_type{});
    // the sequence's last rows, which nothing behind them adds to
    if (stop == end && live) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        const long long t = end - (W - 1) + j;
        if (t >= from && t < own) put8(dxb + t * a.D, open[j]);
      }
    }
  }
  if (a.zero_rows && a.cu && live) {   // the run's rows behind the last sequence
    const long long last = bound(a.N);
    const float none[8] = {};
    for (long long t = last > t0 ? last : t0; t < t1; ++t) put8(dxb + t * a.D, none);
  }
  if (live && (a.dweight || a.dbias)) {
    float* out = a.partial + (size_t)r * (W + 1) * a.D + c;
#pragma unroll
    for (int j = 0; j < W; ++j) put8(out + (size_t)j * a.D, dw[j]);
    put8(out + (size_t)W * a.D, db);
  }
}

// Adds up the runs' rows of [W + 1][D] sums: 16 threads of 4 columns, 16 slices of the runs.
template <typename T>
__global__ __launch_bounds__(256) void conv_sums_kernel(const float* __restrict__ partial, int runs, int W, int D,
                                                        T* __restrict__ dweight, T* __restrict__ dbias) {
  __shared__ f32x4 sm[16][16];
  const int cl = threadIdx.x & 15, sl = threadIdx.x >> 4;
  const long long c = (long long)blockIdx.x * 64 + 4 * cl;   // of (W + 1) D columns: the taps, then the bias
  const long long n = (long long)(W + 1) * D;
  f32x4 acc = zero4();
  if (c < n) {
    const float* p = partial + c;
    int i = sl;
    for (; i + 48 < runs; i += 64) {
      f32x4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const f32x4*>(p + (size_t)(i + 16 * u) * n);
      acc += (x[0] + x[1]) + (x[2] + x[3]);
    }
    for (; i < runs; i += 16) acc += *reinterpret_cast<const f32x4*>(p + (size_t)i * n);
  }
  sm[sl][cl] = acc;
  __syncthreads();
#pragma unroll
  for (int off = 8; off > 0; off >>= 1) {
    if (sl < off) sm[sl][cl] += sm[sl + off][cl];
    __syncthreads();
  }
  if (sl == 0 && c < n) {
    const f32x4 s = sm[0][cl];
    const int j = (int)(c / D), ch = (int)(c - (long long)j * D);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (j < W) {
        if (dweight) dweight[(size_t)(ch + i) * W + j] = from_f<T>(s[i]);
      } else if (dbias) {
        dbias[ch + i] = from_f<T>(s[i]);
      }
    }
  }
}

// Tokens of a run: longer ones repeat less (the W - 1 rows behind them, the taps, a row
// of sums), shorter ones give the chip more waves.  2048 waves are what it holds of this
// kernel.  Both launches, four taps, bf16, 16384 x 8192, 8192 x 8192, 4096 x 4096 and
// 1000 x 8192: 170, 92, 31, 25 us; runs twice as long 190, 102, 30, 22; half as long 179,
// 100, 41, 32.  Never less than 4 (100 x 512 in fp32: 7 us, with 8 10.5).
int run_of(const ConvBwdArgs& a) {
  const int cblocks = (a.D / 8 + 63) / 64;
  const long long units = (long long)a.B * a.T * cblocks;
  long long run = (units / 2048 + 3) / 4 * 4;
  return (int)(run < 4 ? 4 : run > 128 ? 128 : run);
}

template <typename T, int W>
hipError_t launch_w(const ConvBwdArgs& a, hipStream_t s) {
  const long long total = (long long)a.B * a.T;
  const int cblocks = (a.D / 8 + 63) / 64, run = run_of(a);
  const int runs = (int)((total + run - 1) / run);
  if (runs > 0) {
    const dim3 grid((unsigned)((long long)runs * cblocks)), block(64);
    const int lanes = a.norm_sections > 0 ? a.norm_dim / 8 : 0;
    if (lanes == 16) hipLaunchKernelGGL((conv_bwd_kernel<T, W, 16>), grid, block, 0, s, a, run, cblocks);
    else if (lanes == 8) hipLaunchKernelGGL((conv_bwd_kernel<T, W, 8>), grid, block, 0, s, a, run, cblocks);
    else hipLaunchKernelGGL((conv_bwd_kernel<T, W, 0>), grid, block, 0, s, a, run, cblocks);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (!a.dweight && !a.dbias) return hipSuccess;
  const long long n = (long long)(W + 1) * a.D;
  hipLaunchKernelGGL((conv_sums_kernel<T>), dim3((unsigned)((n + 63) / 64)), dim3(256), 0, s, a.partial, runs, W, a.D,
                     reinterpret_cast<T*>(a.dweight), reinterpret_cast<T*>(a.dbias));
  return hipGetLastError();
}

template <typename T>
hipError_t launch_io(const ConvBwdArgs& a, hipStream_t s) {
  if (a.W == 2) return launch_w<T, 2>(a, s);
  if (a.W == 3) return launch_w<T, 3>(a, s);
  return launch_w<T, 4>(a, s);
}

}  // namespace

size_t conv_bwd_bytes(const ConvBwdArgs& a) {
  const long long total = (long long)a.B * a.T;
  if (total == 0 || (!a.dweight && !a.dbias)) return 0;
  const int run = run_of(a);
  return (size_t)((total + run - 1) / run) * (a.W + 1) * a.D * sizeof(float);
}

hipError_t launch_conv_bwd(const ConvBwdArgs& a, hipStream_t s) {
  return a.bf16 ? launch_io<bf16_t>(a, s) : launch_io<float>(a, s);
}

}  // namespace gdn
