// Short causal depthwise convolution in front of a recurrent mixer, gfx950:
// prompts (dense or packed) and single tokens over a pool of states.
//
//   c_t = bias + sum_{j < W} w_j u_{t - W + 1 + j},   W = 2 .. 4,
//
// u being the sequence's rows behind the W - 1 rows of its state; then
// optionally silu, and for prompts optionally an L2 norm over each head of
// the leading sections (the q and k of a delta-rule layer), which needs the
// head's channels only and so costs a few in-row DPP additions here instead of
// another pass over memory.
//
// Memory-bound: 2 elements moved per value and 2 W + ~6 operations.  A lane
// owns 8 consecutive channels (16 bytes of bf16) and walks down a run of
// tokens with the last W - 1 rows in registers, so each row is read once (the
// rows in front of a run a second time, from L2); a wave covers 512 channels
// and its loads and stores are whole 1 KiB pieces of a row.  Nothing is shared
// between waves: no LDS, no barriers.  Sums are fp32; the result is rounded
// once to the io type.
//
// Measured: 16001 packed tokens x 8192 channels, bf16, with norms: 524 MB in 107 us,
// 4.9 TB/s (a large copy 5.1); 2048 tokens 16 us; 100 tokens 5.0 us.
// Steps: 256 rows x 4 tokens x 8192 channels 59 MB in 11 us, 5.2 TB/s (rows and
// states partly from the caches); one row 3 us, a launch.

#include "gdn_device.h"
#include "mixer_launch.h"
#include "rows8.h"

namespace gdn {

namespace {

using namespace rows8;

// What a lane needs of its 8 channels: the taps, the bias, and where results go.
template <typename T, int W>
struct Lane {
  float w[W][8], bias[8];
  T* out;               // of the lane's section, at the lane's channel; row r is `width` elements further
  long long width;
  bool norm;

  __device__ __forceinline__ void init(const ConvArgs& a, int c) {
    const T* wp = reinterpret_cast<const T*>(a.weight) + (size_t)c * W;
    float flat[8 * W];
#pragma unroll
    for (int i = 0; i < W; ++i) {
      Raw8<T> r;
      r.load(wp + 8 * i);
      float f[8];
      r.get(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) flat[8 * i + e] = f[e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = flat[e * W + j];
#pragma unroll
    for (int e = 0; e < 8; ++e) bias[e] = 0.f;
    if (a.bias) {
      Raw8<T> r;
      r.load(reinterpret_cast<const T*>(a.bias) + c);
      r.get(bias);
    }
    const int sec = (c >= a.end[0]) + (c >= a.end[1]);
    const int lo = sec == 0 ? 0 : (sec == 1 ? a.end[0] : a.end[1]);
    const int hi = sec == 0 ? a.end[0] : (sec == 1 ? a.end[1] : a.end[2]);
    T* base = reinterpret_cast<T*>(sec == 0 ? a.out[0] : (sec == 1 ? a.out[1] : a.out[2]));
    width = hi - lo;
    out = base + (c - lo);
    norm = sec < a.norm_sections;
  }
};

// One value row: taps over rows[0 .. W - 1] (oldest first), then the epilogue.
// NORM: lanes of a head, or 0.
template <typename T, int W, int NORM>
__device__ __forceinline__ void emit(const Lane<T, W>& L, const float (&rows)[W][8], int silu, float eps,
                                     long long row) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float s = L.bias[e];
#pragma unroll
    for (int j = 0; j < W; ++j) s = fmaf(L.w[j][e], rows[j][e], s);
    y[e] = s;
  }
  if (silu) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = silu_f(y[e]);
  }
  if constexpr (NORM != 0) {
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) q = fmaf(y[e], y[e], q);
    q = head_sum<NORM>(q) + eps;   // the same in all lanes of a head
    // Squares that leave fp32's range (or its normal numbers, where the reciprocal
    // root takes 0): once more from the head times a power of two, eps times its square.
    if (L.norm && !(q >= 0x1p-100f && q <= 0x1p100f)) {
      const float k = q < 1.0f ? 0x1p100f : 0x1p-70f;
      q = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] *= k;
        q = fmaf(y[e], y[e], q);
      }
      q = head_sum<NORM>(q) + eps * k * k;
    }
    const float f = L.norm ? __builtin_amdgcn_rsqf(q) : 1.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] *= f;
  }
  put8(L.out + row * L.width, y);
}

// Prompts.  A wave handles 512 channels of a run of `run` consecutive packed
// tokens.  Sequences restart inside a run; the wave in whose run a sequence
// starts computes its first W - 1 tokens even where they pass the run's end
// (the next run leaves them out), so it alone reads the sequence's state and
// can write the new one in place.
template <typename T, int W, int NORM>
__global__ __launch_bounds__(64) void conv_fwd_kernel(ConvArgs a, int run, int runs, int cblocks) {
  constexpr int U = 4;   // rows loaded together
  const int lane = threadIdx.x;
  const int r = blockIdx.x / cblocks;
  const int c = ((blockIdx.x - r * cblocks) * 64 + lane) * 8;
  const bool live = c < a.D;
  const long long total = (long long)a.B * a.T;
  const long long t0 = (long long)r * run;
  const long long t1 = t0 + run < total ? t0 + run : total;
  const int cc = live ? c : 0;

  int s;   // first sequence that starts in the run
  if (a.cu) {
    s = __builtin_amdgcn_readfirstlane(first_seq_from(a.cu, a.N, t0, lane));
  } else {
    s = a.T > 0 ? (int)((t0 + a.T - 1) / a.T) : 0;
  }
  auto bound = [&](int n) -> long long {   // clamped boundary n
    if (!a.cu) return (long long)n * a.T;
    const long long v = (long long)a.cu[n];
    return v < 0 ? 0 : (v > total ? total : v);
  };

  Lane<T, W> L;
  L.init(a, cc);
  const T* xb = reinterpret_cast<const T*>(a.x.p) + cc;
  auto row_of = [&](int n, long long start, long long t) -> const T* {   // x at packed token t of sequence n
    return a.cu ? xb + t * a.x.token : xb + (long long)n * a.x.batch + (t - start) * a.x.token;
  };

  float win[W - 1][8];   // the last W - 1 rows
  auto walk = [&](int n, long long start, long long from, long long to) {
    const T* p = row_of(n, start, from);
    for (long long t = from; t < to; t += U) {
      Raw8<T> raw[U];
      const bool full = t + U <= to;   // uniform
      if (full) {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u].load(p + u * a.x.token);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) raw[u].load(p + (t + u < to ? u : 0) * a.x.token);
      }
      p += U * a.x.token;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (full || t + u < to) {
          float rows[W][8];
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) rows[j][e] = win[j][e];
          raw[u].get(rows[W - 1]);
          if (live) emit<T, W, NORM>(L, rows, a.silu, a.eps, t + u);
#pragma unroll
          for (int j = 0; j < W - 1; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) win[j][e] = rows[j + 1][e];
        }
      }
    }
  };

  // the sequence that began before the run: its tokens from W - 1 on
  if (s > 0) {
    const long long start = bound(s - 1);
    long long end = bound(s);
    const long long from = start + W - 1 > t0 ? start + W - 1 : t0;
    end = end < t1 ? end : t1;
    if (start < t0 && from < end) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        Raw8<T> raw;
        raw.load(row_of(s - 1, start, from - (W - 1) + j));
        raw.get(win[j]);
      }
      walk(s - 1, start, from, end);
    }
  }
  const bool last_run = r == runs - 1;
  for (; s < a.N; ++s) {
    const long long start = bound(s);
    if (start >= t1 && !(last_run && start == total)) break;
    if (start < t0) continue;   // boundaries out of order
    long long end = bound(s + 1);
    end = end < start ? start : end;
    T* st = nullptr;
    if (a.state) {
      const int slot = a.idx ? a.idx[s] : s;
      if (slot >= 0 && slot < a.pool)
        st = reinterpret_cast<T*>(a.state) + (size_t)slot * (W - 1) * a.D + cc;
    }
    const bool cont = st && a.has && a.has[s] != 0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
#pragma unroll
      for (int e = 0; e < 8; ++e) win[j][e] = 0.f;
      if (cont) {
        Raw8<T> raw;
        raw.load(st + (size_t)j * a.D);
        raw.get(win[j]);
      }
    }
    long long to = start + W - 1 > t1 ? start + W - 1 : t1;
    to = to < end ? to : end;
    walk(s, start, start, to);
    if (st && live) {
      if (to < end) {   // the rest belongs to later runs: its last rows straight from x
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          Raw8<T> raw;
          raw.load(row_of(s, start, end - (W - 1) + j));
          raw.get(win[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j) put8(st + (size_t)j * a.D, win[j]);
    }
  }
}

// Single tokens: a lane takes 8 channels of one batch row through its TT
// tokens; all loads are issued before the first product.
template <typename T, int W, int TT>
__global__ __launch_bounds__(64) void conv_step_kernel(ConvArgs a, int cblocks) {
  const int b = blockIdx.x / cblocks;
  const int c = ((blockIdx.x - b * cblocks) * 64 + threadIdx.x) * 8;
  if (c >= a.D) return;
  const int slot = a.idx ? a.idx[b] : b;
  const bool valid = slot >= 0 && slot < a.pool;
  T* st = reinterpret_cast<T*>(a.state) + (size_t)(valid ? slot : 0) * (W - 1) * a.D + c;
  Raw8<T> raw[W - 1 + TT];
  if (valid) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) raw[j].load(st + (size_t)j * a.D);
  }
  const T* xb = reinterpret_cast<const T*>(a.x.p) + (long long)b * a.x.batch + c;
#pragma unroll
  for (int t = 0; t < TT; ++t) raw[W - 1 + t].load(xb + t * a.x.token);
  Lane<T, W> L;
  L.init(a, c);
  if (!valid) {   // the pool is not touched
    const float zero[8] = {};
#pragma unroll
    for (int t = 0; t < TT; ++t) put8(L.out + ((long long)b * TT + t) * L.width, zero);
    return;
  }
  float rows[W - 1 + TT][8];
#pragma unroll
  for (int j = 0; j < W - 1 + TT; ++j) raw[j].get(rows[j]);
#pragma unroll
  for (int t = 0; t < TT; ++t) {
    float in[W][8];
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) in[j][e] = rows[t + j][e];
    emit<T, W, 0>(L, in, a.silu, 0.f, (long long)b * TT + t);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) put8(st + (size_t)j * a.D, rows[TT + j]);
}

template <typename T, int W>
hipError_t fwd_w(const ConvArgs& a, hipStream_t s, int run, int runs, int cblocks) {
  const dim3 grid((unsigned)((long long)runs * cblocks)), block(64);
  const int lanes = a.norm_sections > 0 ? a.norm_dim / 8 : 0;
  if (lanes == 16) hipLaunchKernelGGL((conv_fwd_kernel<T, W, 16>), grid, block, 0, s, a, run, runs, cblocks);
  else if (lanes == 8) hipLaunchKernelGGL((conv_fwd_kernel<T, W, 8>), grid, block, 0, s, a, run, runs, cblocks);
  else hipLaunchKernelGGL((conv_fwd_kernel<T, W, 0>), grid, block, 0, s, a, run, runs, cblocks);
  return hipGetLastError();
}

template <typename T, int W>
hipError_t step_w(const ConvArgs& a, hipStream_t s, int cblocks) {
  const dim3 grid((unsigned)((long long)a.B * cblocks)), block(64);
  switch (a.T) {
    case 1: hipLaunchKernelGGL((conv_step_kernel<T, W, 1>), grid, block, 0, s, a, cblocks); break;
    case 2: hipLaunchKernelGGL((conv_step_kernel<T, W, 2>), grid, block, 0, s, a, cblocks); break;
    case 3: hipLaunchKernelGGL((conv_step_kernel<T, W, 3>), grid, block, 0, s, a, cblocks); break;
    default: hipLaunchKernelGGL((conv_step_kernel<T, W, 4>), grid, block, 0, s, a, cblocks); break;
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_conv_fwd(const ConvArgs& a, hipStream_t s) {
  const long long total = (long long)a.B * a.T;
  if (a.N == 0 || (total == 0 && !a.state)) return hipSuccess;
  const int cblocks = (a.D / 8 + 63) / 64;
  // Longer runs repeat less (the taps, and the W - 1 rows in front), shorter ones
  // give the chip more waves: the shortest of 4, 8, 16 tokens that makes at most 4096
  // (8192 channels, W = 4, runs of 4 / 8 / 16: 100 tokens 5.0 / 6.4 / 9.4 us, 700
  // 8.5 / 9.3 / 11.3, 2048 17.1 / 16.2 / 17.4, 4096 28.7 / 28.1 / 26.4; of 32 and 64
  // for 16001 tokens 110 and 111, of 16 109).
  const long long units = total * cblocks;
  const int run = units <= 4 * 4096 ? 4 : units <= 8 * 4096 ? 8 : 16;
  const int runs = total > 0 ? (int)((total + run - 1) / run) : 1;
  if (a.bf16) {
    if (a.W == 2) return fwd_w<bf16_t, 2>(a, s, run, runs, cblocks);
    if (a.W == 3) return fwd_w<bf16_t, 3>(a, s, run, runs, cblocks);
    return fwd_w<bf16_t, 4>(a, s, run, runs, cblocks);
  }
  if (a.W == 2) return fwd_w<float, 2>(a, s, run, runs, cblocks);
  if (a.W == 3) return fwd_w<float, 3>(a, s, run, runs, cblocks);
  return fwd_w<float, 4>(a, s, run, runs, cblocks);
}

hipError_t launch_conv_step(const ConvArgs& a, hipStream_t s) {
  const int cblocks = (a.D / 8 + 63) / 64;
  if (a.bf16) {
    if (a.W == 2) return step_w<bf16_t, 2>(a, s, cblocks);
    if (a.W == 3) return step_w<bf16_t, 3>(a, s, cblocks);
    return step_w<bf16_t, 4>(a, s, cblocks);
  }
  if (a.W == 2) return step_w<float, 2>(a, s, cblocks);
  if (a.W == 3) return step_w<float, 3>(a, s, cblocks);
  return step_w<float, 4>(a, s, cblocks);
}

}  // namespace gdn
