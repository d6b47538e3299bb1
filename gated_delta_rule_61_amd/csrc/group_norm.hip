// Norm of the groups of a token's channels (the heads of a recurrent mixer),
// with an activation or an output gate, and its gradients, gfx950.  Per token
// and group of d channels
//
//   n = (x - mean) r,  r = 1 / sqrt(var + eps)    (rms: n = x / sqrt(mean(x^2) + eps))
//   a = n w + b,       y = a act(z) with a gate z, else act(a)
//
// and, from the gradient of y,
//
//   da = dy act(z)  (no gate: dy act'(a)),  dz = dy a act'(z),  dn = da w
//   dx = r (dn - mean(dn) - n mean(dn n))         (rms: without mean(dn))
//   dw = sum over the tokens (and groups that share w) of da n,  db of da
//
// Memory-bound: three rows of C channels forward (x, z, y), five backward
// (x, z, dy, dx, dz) against 10 and 25 operations a channel.  16384 tokens of 16
// groups of 128 in bf16: 38 us forward (201 MB at 5.3 TB/s), 68 us backward (337 MB at
// 4.9 TB/s) and 5 for the sums of the weights' gradients; a large copy reaches 5.2
// TB/s.  One token: 2.6 us, a launch.
//
// A lane owns 8 consecutive channels (16 bytes of bf16); LPG lanes of a wave hold a group,
// so the sums are in-register: squares of x - mean, not differences of sums.
// The gradient computes n again from x: nothing is kept from the forward pass.
// Groups above 1024 channels take a whole work-group.  A thread keeps its
// channels (w, b, and the sums of dw and db stay in registers) and walks over
// the tokens, the next token's rows in flight; the sums of a work-group's
// threads leave as one row of a workspace, which a second launch adds up in a
// fixed order: the same bits in every run.

#include "gdn_device.h"
#include "mixer_launch.h"
#include "rows8.h"

namespace gdn {

namespace {

constexpr int TPB = 256;

using namespace rows8;

// Sum over the LPG threads of a group, in every one of them.
template <int LPG>
__device__ __forceinline__ float group_sum(float x, float* sm) {
  x += dpp_f<0xB1>(x);
  x += dpp_f<0x4E>(x);
  if constexpr (LPG >= 8) x += dpp_f<0x141>(x);
  if constexpr (LPG >= 16) x += dpp_f<0x140>(x);
  if constexpr (LPG >= 32) x += __shfl_xor(x, 16, 64);
  if constexpr (LPG >= 64) x += __shfl_xor(x, 32, 64);
  if constexpr (LPG == TPB) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) sm[w] = x;
    __syncthreads();
    x = (sm[0] + sm[1]) + (sm[2] + sm[3]);
    __syncthreads();
  }
  return x;
}

__device__ __forceinline__ float sigmoid_f(float a) { return __builtin_amdgcn_rcpf(1.0f + __expf(-a)); }

// act and its slope; kind 0 none, 1 silu, 2 sigmoid
__device__ __forceinline__ float act_f(float a, int kind) {
  const float p = sigmoid_f(a);
  return kind == 0 ? a : kind == 1 ? a * p : p;
}
// 1 - p = e^-a p: the difference keeps nothing of it from a = 17 on.  (e^-a may be infinite,
// where p is 0.)
__device__ __forceinline__ void act_slope(float a, int kind, float& f, float& df) {
  const float e = __expf(-a);
  const float p = __builtin_amdgcn_rcpf(1.0f + e);
  const float q = p * (fminf(e, 3.4028235e38f) * p);
  f = kind == 0 ? a : kind == 1 ? a * p : p;
  df = kind == 0 ? 1.0f : kind == 1 ? fmaf(a, q, p) : q;
}

// One group's statistics: x becomes n, the return value is r.  inv_d = 1 / d.
template <int LPG, int NV>
__device__ __forceinline__ float normalise(float (&x)[NV][8], const bool (&on)[NV], bool rms, float eps, float inv_d,
                                           float* sm) {
  float k = 1.0f;
  auto times = [&](float f) {
    k *= f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] *= f;
  };
  auto sum = [&]() -> float {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += x[v][e];
    return group_sum<LPG>(s, sm);
  };
  auto pass = [&](float s) -> float {   // centres x with its sum s, returns the mean square + eps
    if (!rms) {
      const float mean = s * inv_d;
#pragma unroll
      for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[v][e] = on[v] ? x[v][e] - mean : 0.f;
    }
    float q = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
      for (int e = 0; e < 8; ++e) q = fmaf(x[v][e], x[v][e], q);
    return fmaf(group_sum<LPG>(q, sm), inv_d, eps * k * k);   // k * k alone may pass fp32's largest number
  };
  // What leaves fp32's range, or its normal numbers, where the reciprocal root takes 0, is
  // taken from the group times a power of two, eps times its square (the same in all
  // threads of a group).  The sum, before anything is made from it: below 2^102 the mean is
  // less than half a step of fp32's largest numbers, so x - mean is finite.  Then the
  // squares: times 2^-80, 2^13 of any size have room.
  float s = 0.f;
  if (!rms) {
    s = sum();
    if (!(fabsf(s) <= 0x1p102f)) {
      times(0x1p-80f);
      s = sum();
    }
  }
  float q = pass(s);
  if (!(q >= 0x1p-100f && q <= 0x1p100f)) {
    times(q < 1.0f ? 0x1p100f : 0x1p-80f);
    q = pass(rms ? 0.f : sum());
  }
  const float r = __builtin_amdgcn_rsqf(q);
#pragma unroll
  for (int v = 0; v < NV; ++v)
#pragma unroll
    for (int e = 0; e < 8; ++e) x[v][e] *= r;
  return r * k;
}

// Where a thread works: its group's channels of every `step`-th token from `row` on.
// LPG threads a group, NV vectors of 8 channels each.
template <int LPG, int NV>
struct Place {
  int row, group, cl;
  bool live;
  bool on[NV];
  __device__ __forceinline__ Place(const GroupNormArgs& a, int step) {
    const unsigned id = blockIdx.x * TPB + threadIdx.x;
    const unsigned per = (unsigned)a.G * LPG;   // threads a token
    row = (int)(id / per);
    const unsigned c = id - (unsigned)row * per;
    group = (int)(c / LPG);
    cl = (int)(c % LPG);
    live = row < step;
#pragma unroll
    for (int v = 0; v < NV; ++v) on[v] = live && 8 * (cl + LPG * v) < a.d;
  }
  __device__ __forceinline__ int chan(int v) const { return 8 * (cl + LPG * v); }   // within the group
};

template <int LPG, int NV>
__device__ __forceinline__ void load_weights(const GroupNormArgs& a, const Place<LPG, NV>& p, const void* src,
                                             float none, float (&w)[NV][8]) {
#pragma unroll
  for (int v = 0; v < NV; ++v) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[v][e] = none;
    if (src && p.on[v]) {
      const size_t at = (a.shared ? 0 : (size_t)p.group * a.d) + p.chan(v);
      if (a.w_bf16) {
        Raw8<bf16_t> r;
        r.load(reinterpret_cast<const bf16_t*>(src) + at);
        r.get(w[v]);
      } else {
        Raw8<float> r;
        r.load(reinterpret_cast<const float*>(src) + at);
        r.get(w[v]);
      }
    }
  }
}

// A token's row of a strided operand.
template <typename T>
__device__ __forceinline__ const T* row_of(const Rows& r, int row, int Tlen) {
  const int b = row / Tlen;
  return reinterpret_cast<const T*>(r.p) + (long long)b * r.batch + (long long)(row - b * Tlen) * r.token;
}

template <typename T, int LPG, int NV>
__global__ __launch_bounds__(TPB) void group_norm_fwd_kernel(GroupNormArgs a, int step) {
  __shared__ float sm[4];
  const Place<LPG, NV> p(a, step);
  float w[NV][8], bias[NV][8];
  load_weights(a, p, a.weight, 1.0f, w);
  load_weights(a, p, a.bias, 0.0f, bias);
  const int rows = a.B * a.T;
  const float inv_d = 1.0f / (float)a.d;
  const size_t C = (size_t)a.G * a.d;
  const int c0 = p.group * a.d;
  const bool gated = a.z.p != nullptr;
  Raw8<T> xr[NV], zr[NV];
  auto fetch = [&](int row) {
    const T* xp = row_of<T>(a.x, row, a.T) + c0;
    const T* zp = gated ? row_of<T>(a.z, row, a.T) + c0 : nullptr;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      xr[v] = {};
      zr[v] = {};
      if (p.on[v]) {
        xr[v].load(xp + p.chan(v));
        if (gated) zr[v].load(zp + p.chan(v));
      }
    }
  };
  int row = p.live ? p.row : rows;
  if (row < rows) fetch(row);
  for (; row < rows; row += step) {
    float x[NV][8], z[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      xr[v].get(x[v]);
      zr[v].get(z[v]);
    }
    if (row + step < rows) fetch(row + step);
    normalise<LPG, NV>(x, p.on, a.rms != 0, a.eps, inv_d, sm);
    T* yp = reinterpret_cast<T*>(a.y) + (size_t)row * C + c0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = fmaf(x[v][e], w[v][e], bias[v][e]);
        x[v][e] = gated ? n * act_f(z[v][e], a.act) : act_f(n, a.act);
      }
      if (p.on[v]) put8_nt(yp + p.chan(v), x[v]);
    }
  }
}

// WG: whether dw or db are wanted.
template <typename T, int LPG, int NV, bool WG>
__global__ __launch_bounds__(TPB) void group_norm_bwd_kernel(GroupNormArgs a, int step) {
  __shared__ float sm[4];
  __shared__ __attribute__((aligned(16))) float sums[WG && LPG <= 64 ? 4 : 1][WG && LPG <= 64 ? LPG * 8 * NV : 1];
  const Place<LPG, NV> p(a, step);
  float w[NV][8], bias[NV][8], dw[NV][8] = {}, db[NV][8] = {};
  load_weights(a, p, a.weight, 1.0f, w);
  load_weights(a, p, a.bias, 0.0f, bias);
  const int rows = a.B * a.T;
  const float inv_d = 1.0f / (float)a.d;
  const size_t C = (size_t)a.G * a.d;
  const int c0 = p.group * a.d;
  const bool gated = a.z.p != nullptr;
  Raw8<T> xr[NV], zr[NV], gr[NV];
  auto fetch = [&](int row) {
    const T* xp = row_of<T>(a.x, row, a.T) + c0;
    const T* zp = gated ? row_of<T>(a.z, row, a.T) + c0 : nullptr;
    const T* gp = row_of<T>(a.dout, row, a.T) + c0;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      xr[v] = {};
      zr[v] = {};
      gr[v] = {};
      if (p.on[v]) {
        xr[v].load(xp + p.chan(v));
        if (gated) zr[v].load(zp + p.chan(v));
        gr[v].load(gp + p.chan(v));
      }
    }
  };
  int row = p.live ? p.row : rows;
  if (row < rows) fetch(row);
  for (; row < rows; row += step) {
    float x[NV][8], z[NV][8], g[NV][8];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      xr[v].get(x[v]);
      zr[v].get(z[v]);
      gr[v].get(g[v]);
    }
    if (row + step < rows) fetch(row + step);
    const float r = normalise<LPG, NV>(x, p.on, a.rms != 0, a.eps, inv_d, sm);
    const size_t at = (size_t)row * C + c0;
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = fmaf(x[v][e], w[v][e], bias[v][e]);
        float f, df;
        act_slope(gated ? z[v][e] : n, a.act, f, df);
        z[v][e] = g[v][e] * n * df;
        const float da = g[v][e] * (gated ? f : df);
        if constexpr (WG) {
          dw[v][e] = fmaf(da, x[v][e], dw[v][e]);
          db[v][e] += da;
        }
        const float dn = da * w[v][e];
        g[v][e] = dn;
        s1 += dn;
        s2 = fmaf(dn, x[v][e], s2);
      }
      if (gated && p.on[v]) put8_nt(reinterpret_cast<T*>(a.dz) + at + p.chan(v), z[v]);
    }
    s2 = group_sum<LPG>(s2, sm) * inv_d;
    s1 = a.rms ? 0.f : group_sum<LPG>(s1, sm) * inv_d;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[v][e] = r * (g[v][e] - s1 - x[v][e] * s2);
      if (p.on[v]) put8_nt(reinterpret_cast<T*>(a.dx) + at + p.chan(v), x[v]);
    }
  }
  if constexpr (WG) {
    // one row of sums: [2][d] a work-group where the groups share their weights (a group
    // wider than a wave has a work-group to itself), else [2][C] for each of the `step`
    // walks over the tokens
    if (a.shared && LPG <= 64) {
      const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
#pragma unroll
      for (int part = 0; part < 2; ++part) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float s = part ? db[v][e] : dw[v][e];
#pragma unroll
            for (int off = LPG; off < 64; off <<= 1) s += __shfl_xor(s, off, 64);
            if (lane < LPG) sums[wave][8 * (lane + LPG * v) + e] = s;
          }
        __syncthreads();
        float* out = a.partial + ((size_t)blockIdx.x * 2 + part) * a.d;
        for (int c = threadIdx.x; c < a.d; c += TPB) out[c] = (sums[0][c] + sums[1][c]) + (sums[2][c] + sums[3][c]);
        __syncthreads();
      }
    } else if (p.live) {
      const size_t n = a.shared ? (size_t)a.d : C;
      const size_t prow = a.shared ? (size_t)blockIdx.x : (size_t)p.row;
      float* out = a.partial + prow * 2 * n + (a.shared ? 0 : c0);
#pragma unroll
      for (int v = 0; v < NV; ++v)
        if (p.on[v]) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            *reinterpret_cast<f32x4*>(out + p.chan(v) + 4 * h) =
                f32x4{dw[v][4 * h], dw[v][4 * h + 1], dw[v][4 * h + 2], dw[v][4 * h + 3]};
            *reinterpret_cast<f32x4*>(out + n + p.chan(v) + 4 * h) =
                f32x4{db[v][4 * h], db[v][4 * h + 1], db[v][4 * h + 2], db[v][4 * h + 3]};
          }
        }
    }
  }
}

// Adds up `count` rows of [2][n] sums: 16 threads of 4 columns, 64 slices of the rows.
__global__ __launch_bounds__(1024) void norm_sums_kernel(const float* __restrict__ partial, int count, int n,
                                                         void* dweight, void* dbias, int bf16) {
  __shared__ f32x4 sm[64][16];
  const int cl = threadIdx.x & 15, sl = threadIdx.x >> 4;
  const int c = blockIdx.x * 64 + 4 * cl;   // of 2 n columns: dweight, then dbias
  f32x4 acc = zero4();
  if (c < 2 * n) {
    const float* p = partial + c;
    int i = sl;
    for (; i + 192 < count; i += 256) {
      f32x4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[u] = *reinterpret_cast<const f32x4*>(p + (size_t)(i + 64 * u) * 2 * n);
      acc += (x[0] + x[1]) + (x[2] + x[3]);
    }
    for (; i < count; i += 64) acc += *reinterpret_cast<const f32x4*>(p + (size_t)i * 2 * n);
  }
  sm[sl][cl] = acc;
  __syncthreads();
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) {
    if (sl < off) sm[sl][cl] += sm[sl + off][cl];
    __syncthreads();
  }
  if (sl == 0 && c < 2 * n) {
    const f32x4 s = sm[0][cl];
    void* dst = c < n ? dweight : dbias;
    const int at = c < n ? c : c - n;
    if (dst) {
      if (bf16)
        *reinterpret_cast<uint2*>(reinterpret_cast<bf16_t*>(dst) + at) = uint2{pack_bf2(s[0], s[1]), pack_bf2(s[2], s[3])};
      else
        *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(dst) + at) = s;
    }
  }
}

// Threads and vectors a group of d channels takes: the fewest lanes of a wave with one or
// two vectors each, a work-group where these do not do.  At least four lanes, so groups of
// 8 and 16 channels leave some without any: 16384 tokens of 2048 channels in bf16 take 84
// and 44 us forward, 160 and 85 us backward, where groups of 64 to 2048 take 32 and 60 - 66
// (fp32: 96 and 74, 206 and 150, 71 and 142).
struct Shape {
  int lpg, nv;
};
Shape shape_of(int d) {
  if (d > 1024) return {TPB, d <= 2048 ? 1 : d <= 4096 ? 2 : 4};
  if (d > 512) return {64, 2};
  int l = 4;
  while (l * 8 < d) l *= 2;
  return {l, 1};
}

// Walks over the tokens that run side by side, and the work-groups they take.
struct Walks {
  int step;
  long long blocks;
  long long sums;   // rows of the workspace (the gradient only)
};
Walks walks_of(const GroupNormArgs& a, bool bwd) {
  const Shape sh = shape_of(a.d);
  const long long per = (long long)a.G * sh.lpg, rows = (long long)a.B * a.T;
  // Threads: what the chip holds of these kernels (four, eight waves a SIMD).  16384 tokens
  // of 2048 channels, 2^17, 2^18, 2^19, 2^20 threads, bf16: forward in groups of 16 67, 50,
  // 44, 42 us, of 128 37, 32, 32, 32, of 2048 42, 33, 32, 32; backward 97, 88, 85, 91; 63,
  // 62, 66, 73; 71, 66, 73, 86.  fp32: 69 - 76 and 139 - 161, the fewest threads the fastest
  // backward.  (1001 tokens: 4.4 - 5.5 us forward from 2^18 on; backward with its sums 13 -
  // 20 us from 2^18 on, 11 - 15 with 2^17, whose rows of sums are half as many.)
  const long long want = bwd ? 1 << 18 : 1 << 19;
  long long step = (want + per - 1) / per;
  if (step > rows) step = rows;
  // sums of weights per channel: a walk leaves two rows of them, so it takes four tokens at
  // least (1001 tokens of 16 groups of 80 in fp32: 8.7 us + 5 for the sums; no less in all
  // with two), whichever of the sums is wanted: the size of the workspace tells nothing of that
  if (bwd && !a.shared && (a.dweight || a.dbias) && step > (rows + 3) / 4) step = (rows + 3) / 4;
  Walks w;
  w.step = (int)step;
  w.blocks = (step * per + TPB - 1) / TPB;
  w.sums = a.shared ? w.blocks : step;
  return w;
}

template <typename T, int LPG, int NV>
hipError_t launch_n(const GroupNormArgs& a, hipStream_t s, bool bwd) {
  const Walks w = walks_of(a, bwd);   // no tokens: no walks, and sums of nothing
  const dim3 grid((unsigned)w.blocks), block(TPB);
  if (!bwd) {
    if (w.blocks == 0) return hipSuccess;
    hipLaunchKernelGGL((group_norm_fwd_kernel<T, LPG, NV>), grid, block, 0, s, a, w.step);
    return hipGetLastError();
  }
  const bool sums = a.dweight || a.dbias;
  if (w.blocks > 0) {
    if (sums) hipLaunchKernelGGL((group_norm_bwd_kernel<T, LPG, NV, true>), grid, block, 0, s, a, w.step);
    else hipLaunchKernelGGL((group_norm_bwd_kernel<T, LPG, NV, false>), grid, block, 0, s, a, w.step);
    if (hipError_t e = hipGetLastError()) return e;
  }
  if (!sums) return hipSuccess;
  const int n = a.shared ? a.d : a.G * a.d;
  hipLaunchKernelGGL(norm_sums_kernel, dim3((unsigned)((2LL * n + 63) / 64)), dim3(1024), 0, s, a.partial, (int)w.sums,
                     n, a.dweight, a.dbias, a.w_bf16);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_io(const GroupNormArgs& a, hipStream_t s, bool bwd) {
  const Shape sh = shape_of(a.d);
  switch (sh.lpg) {
    case 4: return launch_n<T, 4, 1>(a, s, bwd);
    case 8: return launch_n<T, 8, 1>(a, s, bwd);
    case 16: return launch_n<T, 16, 1>(a, s, bwd);
    case 32: return launch_n<T, 32, 1>(a, s, bwd);
    case 64: return sh.nv == 1 ? launch_n<T, 64, 1>(a, s, bwd) : launch_n<T, 64, 2>(a, s, bwd);
    default:
      if (sh.nv == 1) return launch_n<T, TPB, 1>(a, s, bwd);
      return sh.nv == 2 ? launch_n<T, TPB, 2>(a, s, bwd) : launch_n<T, TPB, 4>(a, s, bwd);
  }
}

}  // namespace

size_t group_norm_bwd_bytes(const GroupNormArgs& a) {
  const long long rows = (long long)a.B * a.T;
  if (rows == 0 || (!a.dweight && !a.dbias)) return 0;
  return (size_t)walks_of(a, true).sums * 2 * (a.shared ? (size_t)a.d : (size_t)a.G * a.d) * sizeof(float);
}

hipError_t launch_group_norm_fwd(const GroupNormArgs& a, hipStream_t s) {
  return a.bf16 ? launch_io<bf16_t>(a, s, false) : launch_io<float>(a, s, false);
}

hipError_t launch_group_norm_bwd(const GroupNormArgs& a, hipStream_t s) {
  return a.bf16 ? launch_io<bf16_t>(a, s, true) : launch_io<float>(a, s, true);
}

}  // namespace gdn
