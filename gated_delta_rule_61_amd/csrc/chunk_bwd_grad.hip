// The chunk-parallel part of the chunked rule's gradients, gfx950 (chunk_bwd.h has
// the mathematics): dq, dk, dv, dg and dbeta of a chunk from the states, the state
// gradients, Vn and dR that the two scans left.
//
// A work-group is one (chunk, key head): it takes the v-heads that share the key
// head in turn and adds their dq and dk in registers, in order.  Products run
// transposed ([K channels] x [tokens]), so that a lane ends with 8 consecutive
// channels of a token: 16-byte stores, and the dot products with q and k (which
// make dg and dbeta) in registers.  Each wave has 32 channels (K = 64: and half
// the tokens); reductions over V go in blocks of 64 columns, whose tiles (dO, Vn,
// dR, h, dh') pass through LDS once, the next block's in flight in registers.  The
// scores dO Vn^T and dR Vn^T are dealt out to the waves in 16 x 16 blocks, gated
// and masked there and shared through LDS, in the bytes of the tiles that are no
// longer needed.

#include "chunk_bwd.h"
#include "chunk_common.h"

namespace gdn {

namespace {

using namespace bwd;

template <typename C, int D>
struct GradLds {
  static constexpr int T64 = Tile<C, 64>::bytes(BT), TD = Tile<C, D>::bytes(BT);
  // a block of 64 V columns: dO [t][v], Vn^T and dR^T [v][t], h and dh' [v][k];
  // later the scores in the first three, k and q [t][channel] in the last two
  static constexpr int O = 0, VN = T64, DR = 2 * T64, H = 3 * T64, DS = H + TD;
  static constexpr int G = DS + TD;             // G, e^G, e^{G_last - G}, beta of the tokens
  static constexpr int RED = G + 4 * BT * 4;    // dot products [4][4][64], one row for 32 channels
  static constexpr int VDR = RED + 16 * BT * 4; // v . dR [64], <h, dh'> of each wave [4]
  static constexpr int bytes = VDR + BT * 4 + 16;
};

// Vectors of 8 elements that 256 threads move of a [64][COLS] tile.
template <typename T, int COLS> struct Moved {
  static constexpr int N = BT * COLS / 8 / 256;
  Frag<T> f[N];
  static __device__ __forceinline__ int row(int i, int tid) { return (tid + 256 * i) / (COLS / 8); }
  static __device__ __forceinline__ int col(int i, int tid) { return (tid + 256 * i) % (COLS / 8) * 8; }
};

template <typename T, int D, bool GROUPED>
__global__ __launch_bounds__(256) void gdn_bwd_grad_kernel(ChunkBwdArgs a) {
  typedef typename ComputeOf<T>::type C;
  typedef GradLds<C, D> L;
  typedef Tile<C, D> TD;
  typedef Tile<C, 64> T64;
  constexpr int VB = D / 64;          // blocks of V columns
  constexpr int KW = D / 32;          // waves side by side over the channels
  constexpr int NT = KW;              // 16-token blocks of a wave
  extern __shared__ __attribute__((aligned(16))) char lds[];
  float* const sG = reinterpret_cast<float*>(lds + L::G);
  float* const red = reinterpret_cast<float*>(lds + L::RED);
  float* const sVdr = reinterpret_cast<float*>(lds + L::VDR);

  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int kw = w % KW, tb0 = w / KW * NT;   // the wave's channels 32 kw .. and token blocks
  const int Hk = a.f.Hk, HV = a.f.HV, GR = HV / Hk;
  const int NTC = (a.f.T + BT - 1) / BT;
  int slot, jk, c0, nrow;
  if (!intra::slot_of_block(a.nslots, Hk, slot, jk)) return;
  if (!intra::locate_chunk(slot, a.f.cu_seqlens, a.f.chunk_off, a.f.N, a.f.T, NTC, c0, nrow)) return;
  int ns;   // the chunk's sequence (of amax)
  if (a.f.cu_seqlens) {
    int lo = 0, hi = a.f.N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.f.chunk_off[mid] <= slot) lo = mid; else hi = mid;
    }
    ns = lo;
  } else {
    ns = slot / NTC;
  }

  const size_t krow = (size_t)Hk * D, vstride = (size_t)HV * D;
  const T* const qp = reinterpret_cast<const T*>(a.f.q) + (size_t)c0 * krow + (size_t)jk * D;
  const T* const kp = reinterpret_cast<const T*>(a.f.k) + (size_t)c0 * krow + (size_t)jk * D;

  f32x4 dq_sum[GROUPED ? 2 : 1][GROUPED ? NT : 1], dk_sum[GROUPED ? 2 : 1][GROUPED ? NT : 1];
  if constexpr (GROUPED) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t) dq_sum[h][t] = dk_sum[h][t] = zero4();
  }

  for (int r = 0; r < GR; ++r) {
    const int j = jk * GR + r;
    float inv = 1.f, gs = 1.f;
    if (a.amax) gs = grad_scale(a.amax[(size_t)ns * HV + j], inv);
    const size_t cell = (size_t)slot * HV + j;
    const T* const dop = reinterpret_cast<const T*>(a.dout) + (size_t)c0 * vstride + (size_t)j * D;
    const T* const vp = reinterpret_cast<const T*>(a.f.v) + (size_t)c0 * vstride + (size_t)j * D;
    T* const dvp = reinterpret_cast<T*>(a.dv) + (size_t)c0 * vstride + (size_t)j * D;
    const C* const vnp = reinterpret_cast<const C*>(a.vn) + cell * D * BT;
    const C* const drp = reinterpret_cast<const C*>(a.dr) + cell * D * BT;
    const C* const hp = reinterpret_cast<const C*>(a.hs) + cell * D * D;
    const C* const dsp = reinterpret_cast<const C*>(a.ds) + cell * D * D;

    Moved<T, 64> o_in;
    Moved<C, 64> vn_in, dr_in;
    Moved<C, D> h_in, ds_in;
    auto fetch = [&](int vb) {
#pragma unroll
      for (int i = 0; i < o_in.N; ++i) {
        const int t = o_in.row(i, tid), v = 64 * vb + o_in.col(i, tid);
        if (t < nrow) load8(o_in.f[i], dop + (size_t)t * vstride + v);
        else o_in.f[i].zero();
      }
#pragma unroll
      for (int i = 0; i < vn_in.N; ++i) {
        const size_t at = (size_t)(64 * vb + vn_in.row(i, tid)) * BT + vn_in.col(i, tid);
        load8(vn_in.f[i], vnp + at);
        load8(dr_in.f[i], drp + at);
      }
#pragma unroll
      for (int i = 0; i < h_in.N; ++i) {
        const size_t at = (size_t)(64 * vb + h_in.row(i, tid)) * D + h_in.col(i, tid);
        load8(h_in.f[i], hp + at);
        load8(ds_in.f[i], dsp + at);
      }
    };
    fetch(0);
    // the gates: G again from its terms, beta
    if (w == 0) {
      const int tl = lane < nrow ? lane : nrow - 1;
      const float graw = a.f.g ? a.f.g[(size_t)(c0 + tl) * HV + j] : (a.f.g_gamma ? a.f.g_gamma[j] : 0.f);
      const float b = a.f.beta[(size_t)(c0 + tl) * HV + j];
      const float G = intra::wave_incl_scan(lane < nrow ? graw : 0.f, lane);
      const float Gl = __shfl(G, nrow - 1, 64);
      sG[lane] = G;
      sG[BT + lane] = __expf(G);
      sG[2 * BT + lane] = lane < nrow ? __expf(Gl - G) : 0.f;
      sG[3 * BT + lane] = lane < nrow ? b : 0.f;
    }

    f32x4 dq[2][NT], E[2][NT], W[2][NT], M[5];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t) dq[h][t] = E[h][t] = W[h][t] = zero4();
#pragma unroll
    for (int i = 0; i < 5; ++i) M[i] = zero4();
    float hd = 0.f;     // <h, dh'>, this thread's elements
    float vdr = 0.f;    // v . dR of token 16 w + n, this lane's channels

    for (int vb = 0; vb < VB; ++vb) {
      __syncthreads();
#pragma unroll
      for (int i = 0; i < o_in.N; ++i) T64::put(lds + L::O, o_in.row(i, tid), o_in.col(i, tid), widen(o_in.f[i], gs));
#pragma unroll
      for (int i = 0; i < vn_in.N; ++i) {
        T64::put(lds + L::VN, vn_in.row(i, tid), vn_in.col(i, tid), vn_in.f[i]);
        T64::put(lds + L::DR, dr_in.row(i, tid), dr_in.col(i, tid), dr_in.f[i]);
      }
#pragma unroll
      for (int i = 0; i < h_in.N; ++i) {
        TD::put(lds + L::H, h_in.row(i, tid), h_in.col(i, tid), h_in.f[i]);
        TD::put(lds + L::DS, ds_in.row(i, tid), ds_in.col(i, tid), ds_in.f[i]);
        const f32x8 x = values(h_in.f[i]), y = values(ds_in.f[i]);
#pragma unroll
        for (int e = 0; e < 8; ++e) hd = fmaf(x[e], y[e], hd);
      }
      if (vb + 1 < VB) fetch(vb + 1);
      __syncthreads();

#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int r0 = 32 * s + 8 * g;   // the lane's 8 V columns of the block
        Frag<C> hf[2], df[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          hf[h] = TD::col(lds + L::H + TD::pair_cols(kw, n, g) + 32 * s * TD::pitch + h * TD::odd);
          df[h] = TD::col(lds + L::DS + TD::pair_cols(kw, n, g) + 32 * s * TD::pitch + h * TD::odd);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int tb = tb0 + t;
          const Frag<C> of = T64::row8(lds + L::O, 16 * tb + n, r0);
          const Frag<C> rf = T64::col(lds + L::DR + T64::block_cols(tb, n, g) + 32 * s * T64::pitch);
          const Frag<C> vf = T64::col(lds + L::VN + T64::block_cols(tb, n, g) + 32 * s * T64::pitch);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            dq[h][t] = mma(hf[h], of, dq[h][t]);
            E[h][t] = mma(hf[h], rf, E[h][t]);
            W[h][t] = mma(df[h], vf, W[h][t]);
          }
        }
        // scores, transposed: block i of the wave is one of dO Vn^T (0 .. 9) or dR Vn^T
        // (10 .. 19), lower blocks (tb, sb) in the order of tix
#pragma unroll
        for (int i = 0; i < 5; ++i) {
          const int b = w + 4 * i;
          const int m = b >= 10 ? b - 10 : b;
          const int tb = m >= 6 ? 3 : m >= 3 ? 2 : m >= 1 ? 1 : 0, sb = m - tb * (tb + 1) / 2;
          const Frag<C> vf = T64::col(lds + L::VN + T64::block_cols(sb, n, g) + 32 * s * T64::pitch);
          const Frag<C> xf = b >= 10 ? T64::col(lds + L::DR + T64::block_cols(tb, n, g) + 32 * s * T64::pitch)
                                     : T64::row8(lds + L::O, 16 * tb + n, r0);
          M[i] = mma(vf, xf, M[i]);
        }
        // dv of token 16 w + n, and v . dR
        const int t = 16 * w + n;
        if (t < nrow) {
          const f32x8 x = values(T64::col(lds + L::DR + T64::block_cols(w, n, g) + 32 * s * T64::pitch));
          const size_t at = (size_t)t * vstride + 64 * vb + r0;
          Frag<T> vv;
          load8(vv, vp + at);
          const f32x8 y = values(vv);
#pragma unroll
          for (int e = 0; e < 8; ++e) vdr = fmaf(x[e], y[e], vdr);
          store_io8(dvp + at, x * (sG[3 * BT + t] * inv));
        }
      }
    }
    // k and q rows for the products within the chunk, in flight over the barrier
    Moved<T, D> k_in, q_in;
#pragma unroll
    for (int i = 0; i < k_in.N; ++i) {
      const int t = k_in.row(i, tid), c = k_in.col(i, tid);
      if (t < nrow) {
        load8(k_in.f[i], kp + (size_t)t * krow + c);
        load8(q_in.f[i], qp + (size_t)t * krow + c);
      } else {
        k_in.f[i].zero();
        q_in.f[i].zero();
      }
    }
    __syncthreads();
    char* const sK = lds + L::H;
    char* const sQ = lds + L::DS;
    char* const S1 = lds + L::O;    // scale dO Vn^T o Gamma, s <= t
    char* const S2 = lds + L::VN;   // -dR Vn^T o Gamma, s < t
    char* const S3 = lds + L::DR;   // beta_t times that
#pragma unroll
    for (int i = 0; i < k_in.N; ++i) {
      TD::put(sK, k_in.row(i, tid), k_in.col(i, tid), widen(k_in.f[i]));
      TD::put(sQ, q_in.row(i, tid), q_in.col(i, tid), widen(q_in.f[i]));
    }
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int b = w + 4 * i;
      const bool second = b >= 10;
      const int m = second ? b - 10 : b;
      const int tb = m >= 6 ? 3 : m >= 3 ? 2 : m >= 1 ? 1 : 0, sb = m - tb * (tb + 1) / 2;
      const int t = 16 * tb + n, s = 16 * sb + 4 * g;
      const float Gt = sG[t], f = second ? -1.f : a.f.scale;
      const f32x4 Gs = *reinterpret_cast<const f32x4*>(sG + s);
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool keep = second ? s + e < t : s + e <= t;
        x[e] = keep ? f * M[i][e] * __expf(Gt - Gs[e]) : 0.f;
      }
      T64::put4(second ? S2 : S1, t, s, x);
      if (second) T64::put4(S3, t, s, x * sG[3 * BT + t]);
    }
    // the blocks above the diagonal that a 32-wide slab takes in
    for (int i = w; i < 6; i += 4) {
      char* const tile = i / 2 == 0 ? S1 : i / 2 == 1 ? S2 : S3;
      T64::put4(tile, 32 * (i & 1) + n, 32 * (i & 1) + 16 + 4 * g, zero4());
    }
    __syncthreads();

    // row factors, the dot product with k of what crosses the chunk's end
    Frag<C> kf[NT], qf[NT];
    float wi[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = 16 * (tb0 + t) + n;
      kf[t] = TD::row8(sK, tok, 32 * kw + 8 * g);
      qf[t] = TD::row8(sQ, tok, 32 * kw + 8 * g);
      const float ex = sG[BT + tok], ey = sG[2 * BT + tok];
      const f32x8 k8 = values(kf[t]);
      wi[t] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        dq[h][t] = dq[h][t] * (a.f.scale * ex);
        E[h][t] = E[h][t] * -ex;
        W[h][t] = W[h][t] * ey;
#pragma unroll
        for (int e = 0; e < 4; ++e) wi[t] = fmaf(k8[4 * h + e], W[h][t][e], wi[t]);
      }
    }
    // products within the chunk: only slabs that meet entries below the diagonal
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int r0 = 32 * p + 8 * g;
      Frag<C> ka[2], qa[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ka[h] = TD::col(sK + TD::pair_cols(kw, n, g) + 32 * p * TD::pitch + h * TD::odd);
        qa[h] = TD::col(sQ + TD::pair_cols(kw, n, g) + 32 * p * TD::pitch + h * TD::odd);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tb = tb0 + t;
        if (2 * p <= tb) {   // s of the slab up to t
          const Frag<C> s1 = T64::row8(S1, 16 * tb + n, r0), s2 = T64::row8(S2, 16 * tb + n, r0);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            dq[h][t] = mma(ka[h], s1, dq[h][t]);
            E[h][t] = mma(ka[h], s2, E[h][t]);
          }
        }
        if (2 * p + 1 >= tb) {   // t of the slab from s = 16 tb + n on
          const Frag<C> s1 = T64::col(S1 + T64::block_cols(tb, n, g) + 32 * p * T64::pitch), s3 = T64::col(S3 + T64::block_cols(tb, n, g) + 32 * p * T64::pitch);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            W[h][t] = mma(qa[h], s1, W[h][t]);
            W[h][t] = mma(ka[h], s3, W[h][t]);
          }
        }
      }
    }
    // dots over the wave's channels, and the sums of k . E and the rest
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = 16 * (tb0 + t) + n;
      const f32x8 k8 = values(kf[t]), q8 = values(qf[t]);
      float qd = 0.f, ke = 0.f, kW = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          qd = fmaf(q8[4 * h + e], dq[h][t][e], qd);
          ke = fmaf(k8[4 * h + e], E[h][t][e], ke);
          kW = fmaf(k8[4 * h + e], W[h][t][e], kW);
        }
      float d[4] = {qd, ke, kW, wi[t]};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i] += __shfl_xor(d[i], 16, 64);
        d[i] += __shfl_xor(d[i], 32, 64);
        if (g == 0) red[(i * 4 + kw) * BT + tok] = d[i];
      }
      // dk = beta E + W
      const float b = sG[3 * BT + tok];
      f32x4 x[2], y[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        x[h] = dq[h][t] * inv;
        y[h] = (E[h][t] * b + W[h][t]) * inv;
        if constexpr (GROUPED) {
          dq_sum[h][t] += x[h];
          dk_sum[h][t] += y[h];
        }
      }
      if constexpr (!GROUPED) {
        if (tok < nrow) {
          const size_t at = (size_t)(c0 + tok) * krow + (size_t)jk * D + 32 * kw + 8 * g;
          store_io8(reinterpret_cast<T*>(a.dq) + at, both(x[0], x[1]));
          store_io8(reinterpret_cast<T*>(a.dk) + at, both(y[0], y[1]));
        }
      }
    }
    vdr += __shfl_xor(vdr, 16, 64);
    vdr += __shfl_xor(vdr, 32, 64);
    if (g == 0) sVdr[16 * w + n] = vdr;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) hd += __shfl_xor(hd, off, 64);
    if (lane == 0) sVdr[BT + w] = hd;
    __syncthreads();
    if (w == 0) {
      float d[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        d[i] = 0.f;
#pragma unroll
        for (int c = 0; c < KW; ++c) d[i] += red[(i * 4 + c) * BT + lane];
      }
      const float b = sG[3 * BT + lane];
      const bool live = lane < nrow;
      float dG = live ? d[0] + b * d[1] - d[2] : 0.f;
      // at the last row: the state at the chunk's end and its gradient
      float cross = live ? d[3] : 0.f;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) cross += __shfl_xor(cross, off, 64);
      cross += sG[BT + nrow - 1] * ((sVdr[BT] + sVdr[BT + 1]) + (sVdr[BT + 2] + sVdr[BT + 3]));
      // sums from each row to the end
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const float y = __shfl_down(dG, off, 64);
        if (lane + off < 64) dG += y;
      }
      if (live) {
        const size_t at = (size_t)(c0 + lane) * HV + j;
        if (a.dg) reinterpret_cast<T*>(a.dg)[at] = from_f<T>((dG + cross) * inv);
        reinterpret_cast<T*>(a.dbeta)[at] = from_f<T>((sVdr[lane] + d[1]) * inv);
      }
    }
    __syncthreads();   // the gates and dots are written again for the next head
  }
  if constexpr (GROUPED) {
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int tok = 16 * (tb0 + t) + n;
      if (tok < nrow) {
        const size_t at = (size_t)(c0 + tok) * krow + (size_t)jk * D + 32 * kw + 8 * g;
        store_io8(reinterpret_cast<T*>(a.dq) + at, both(dq_sum[0][t], dq_sum[1][t]));
        store_io8(reinterpret_cast<T*>(a.dk) + at, both(dk_sum[0][t], dk_sum[1][t]));
      }
    }
  }
}

template <typename T, int D, bool GROUPED>
hipError_t launch_grad(const ChunkBwdArgs& a, hipStream_t s) {
  typedef GradLds<typename ComputeOf<T>::type, D> L;
  const void* kern = reinterpret_cast<const void*>(gdn_bwd_grad_kernel<T, D, GROUPED>);
  if (L::bytes > 65536)
    if (hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, L::bytes)) return e;
  hipLaunchKernelGGL((gdn_bwd_grad_kernel<T, D, GROUPED>), dim3(intra::intra_blocks(a.nslots, a.f.Hk)), dim3(256),
                     L::bytes, s, a);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_io(const ChunkBwdArgs& a, hipStream_t s) {
  const bool grouped = a.f.HV != a.f.Hk;
  if (a.f.K == 128) return grouped ? launch_grad<T, 128, true>(a, s) : launch_grad<T, 128, false>(a, s);
  return grouped ? launch_grad<T, 64, true>(a, s) : launch_grad<T, 64, false>(a, s);
}

}  // namespace

hipError_t launch_chunk_bwd_grad(const ChunkBwdArgs& a, hipStream_t s) {
  return a.f.bf16 ? launch_io<bf16_t>(a, s) : launch_io<float>(a, s);
}

}  // namespace gdn
