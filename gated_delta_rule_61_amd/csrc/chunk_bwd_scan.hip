// The two sequential parts of the chunked rule's gradients, gfx950 (chunk_bwd.h
// has the mathematics): the states h and new values Vn again, first chunk to
// last, and the state gradients dh' and dR, last chunk to first.  Neither needs
// the other, and every V column of either stands for itself: one launch runs both
// at once, with twice the work-groups of one.
//
// A work-group is one (sequence, v-head, 64 columns, direction): four waves of 16
// columns, whose state (K x 16, fp32) stays in MFMA accumulators.  As in the
// prefill's scan, rows of the A operands are placed so that two accumulators are
// the next product's B operand, without a trip through LDS: K h -> R -> A R ->
// state, and K dh' -> Y -> A^T Y -> state.  The chunk's K (and Q), A (and P), v or
// dO tiles are shared through LDS, in the compute type, rows behind the
// sequence's end as zeros; those of the next chunk are in flight in registers
// meanwhile.  Row fragments are 16-byte reads; K^T, Q^T, A^T, P^T and dO^T come
// from the same tiles by transposing reads.
//
// h and dh' leave as [V][K] rows, Vn and dR transposed ([V][64]): what a lane's
// accumulators hold in order.

#include "chunk_bwd.h"

namespace gdn {

namespace {

using namespace bwd;

// chunk slot's offset of the sequence, its bounds; false when it has no chunks
__device__ __forceinline__ void seq_bounds(const ChunkArgs& a, int ns, int& bos, int& eos) {
  if (a.cu_seqlens) {
    long long b0 = a.cu_seqlens[ns], b1 = a.cu_seqlens[ns + 1];
    b0 = b0 < 0 ? 0 : (b0 > a.T ? a.T : b0);
    b1 = b1 < b0 ? b0 : (b1 > a.T ? a.T : b1);
    bos = (int)b0;
    eos = (int)b1;
  } else {
    bos = ns * a.T;
    eos = bos + a.T;
  }
}

template <typename T, typename C, int D>
struct ScanLds {
  static constexpr int K = 0;
  static constexpr int A = Tile<C, D>::bytes(BT);
  static constexpr int V = A + Tile<C, 64>::bytes(BT);         // v (io type) or dO (compute type)
  static constexpr int G = V + Tile<C, 64>::bytes(BT);         // gate factors: e^G, e^{G_last - G}, beta, e^{G_last}
  static constexpr int Q = G + 4 * BT * 4;                     // backward only
  static constexpr int P = Q + Tile<C, D>::bytes(BT);
  static constexpr int bytes = P + Tile<C, 64>::bytes(BT);
};

// A [64][COLS] tile on its way from global memory to LDS: 256 threads, 8
// consecutive elements each and step.
template <typename T, int COLS> struct Stage {
  static constexpr int N = BT * COLS / 8 / 256;
  Frag<T> f[N];
  // rows `row` elements apart; those at or behind nrow become zeros
  __device__ __forceinline__ void load(const T* p, size_t row, int nrow, int tid) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = (tid + 256 * i) / (COLS / 8), c = (tid + 256 * i) % (COLS / 8) * 8;
      if (r < nrow) load8(f[i], p + (size_t)r * row + c);
      else f[i].zero();
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F&& put, int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) put((tid + 256 * i) / (COLS / 8), (tid + 256 * i) % (COLS / 8) * 8, f[i]);
  }
};

// v tile of the forward direction: the io type, 64 columns
template <typename T> struct VTile;
template <> struct VTile<bf16_t> {
  typedef Tile<f16_t, 64> L;   // 16-bit elements, whatever they are
  static __device__ __forceinline__ void put(char* t, int r, int c, const Frag<bf16_t>& f) {
    *reinterpret_cast<bf16x8*>(t + L::off(r, c)) = f.v;
  }
  // rows perm_row(tb, 4 g) .. + 3 of column 16 w + n
  static __device__ __forceinline__ f32x4 get(const char* t, int tb, int w, int n, int g) {
    const uint2 r = tiles::ld_tr(t + L::off(perm_row(tb, 4 * g + (n >> 2)), 16 * w + 4 * (n & 3)));
    return f32x4{__builtin_bit_cast(float, r.x << 16), __builtin_bit_cast(float, r.x & 0xFFFF0000u),
                 __builtin_bit_cast(float, r.y << 16), __builtin_bit_cast(float, r.y & 0xFFFF0000u)};
  }
};
template <> struct VTile<float> {
  typedef Tile<float, 64> L;
  static __device__ __forceinline__ void put(char* t, int r, int c, const Frag<float>& f) { L::put(t, r, c, f); }
  static __device__ __forceinline__ f32x4 get(const char* t, int tb, int w, int n, int g) {
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = *reinterpret_cast<const float*>(t + L::off(perm_row(tb, 4 * g) + i, 16 * w + n));
    return x;
  }
};

template <typename T, int D>
__global__ __launch_bounds__(256) void gdn_bwd_scan_kernel(ChunkBwdArgs a) {
  typedef typename ComputeOf<T>::type C;
  typedef ScanLds<T, C, D> L;
  typedef Tile<C, D> TK;
  typedef Tile<C, 64> TA;
  constexpr int KS = D / 32, KB = D / 16, NVT = D / 64;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  char* const sK = lds + L::K;
  char* const sA = lds + L::A;
  char* const sV = lds + L::V;
  float* const sG = reinterpret_cast<float*>(lds + L::G);
  char* const sQ = lds + L::Q;
  char* const sP = lds + L::P;

  const int tid = threadIdx.x, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int Hk = a.f.Hk, HV = a.f.HV;

  // Work-group -> (sequence, head, columns, direction).  Ids are dealt round-robin to
  // the 8 XCDs: the work-groups of a (sequence, key head) run next to each other on one,
  // whose L2 they share; the longest sequences first.
  const int GR = HV / Hk, per = GR * NVT * 2;
  const int pos = blockIdx.x >> 3;
  const int unit = (pos / per) * 8 + (blockIdx.x & 7);
  if (unit >= a.f.N * Hk) return;
  const int rem = pos % per;
  const bool back = rem % 2 == 0;
  const int v0 = rem / 2 % NVT * 64;
  const int rank = unit / Hk, jk = unit - rank * Hk, j = jk * GR + rem / (2 * NVT);
  const int ns = a.f.seq_order ? a.f.seq_order[rank] : rank;
  int bos, eos;
  seq_bounds(a.f, ns, bos, eos);
  int NC = (eos - bos + BT - 1) / BT;
  const int slot0 = a.f.chunk_off ? a.f.chunk_off[ns] : ns * ((a.f.T + BT - 1) / BT);
  // only boundaries out of order can reach past the slots
  if (slot0 + NC > a.nslots) NC = a.nslots > slot0 ? a.nslots - slot0 : 0;
  const int vrow = v0 + 16 * w + n;   // the lane's column
  const size_t sbase = (((size_t)ns * HV + j) * D + vrow) * D;

  float inv = 1.f, gs = 1.f;
  if (back && a.amax) gs = grad_scale(a.amax[(size_t)ns * HV + j], inv);

  f32x4 S[KB];
  const float* init = back ? a.dht : a.f.h0;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    S[kb] = zero4();
    if (init) S[kb] = *reinterpret_cast<const f32x4*>(init + sbase + perm_row(kb, 4 * g)) * gs;
  }

  const size_t krow = (size_t)Hk * D, vstride = (size_t)HV * D, arow = (size_t)HV * BT;
  const size_t plane = (size_t)gf_stride((long long)a.f.B * a.f.T);
  const T* const vsrc = reinterpret_cast<const T*>(back ? a.dout : a.f.v) + (size_t)j * D + v0;
  const C* const Ain = reinterpret_cast<const C*>(a.f.Ainv) + (size_t)j * BT;
  const C* const Pin = reinterpret_cast<const C*>(a.f.Aqk) + (size_t)j * BT;
  const float* const GF = reinterpret_cast<const float*>(a.f.GF) + (size_t)j * 4 * plane;

  Stage<T, D> k_in, q_in;
  Stage<C, 64> a_in, p_in;
  Stage<T, 64> v_in;
  float gate_in = 0.f;
  auto fetch = [&](int c) {
    const int c0 = bos + BT * c, nrow = eos - c0 < BT ? eos - c0 : BT;
    const size_t t0 = (size_t)c0;
    k_in.load(reinterpret_cast<const T*>(a.f.k) + (size_t)jk * D + t0 * krow, krow, nrow, tid);
    a_in.load(Ain + t0 * arow, arow, nrow, tid);
    v_in.load(vsrc + t0 * vstride, vstride, nrow, tid);
    if (back) {
      q_in.load(reinterpret_cast<const T*>(a.f.q) + (size_t)jk * D + t0 * krow, krow, nrow, tid);
      p_in.load(Pin + t0 * arow, arow, nrow, tid);
    }
    gate_in = lane < nrow ? GF[(size_t)w * plane + t0 + lane] : 0.f;
  };
  auto place = [&]() {
    k_in.each([&](int r, int col, const Frag<T>& f) { TK::put(sK, r, col, widen(f)); }, tid);
    a_in.each([&](int r, int col, const Frag<C>& f) { TA::put(sA, r, col, f); }, tid);
    sG[tid] = gate_in;
    if (back) {
      v_in.each([&](int r, int col, const Frag<T>& f) { TA::put(sV, r, col, widen(f, gs)); }, tid);
      q_in.each([&](int r, int col, const Frag<T>& f) { TK::put(sQ, r, col, widen(f)); }, tid);
      p_in.each([&](int r, int col, const Frag<C>& f) { TA::put(sP, r, col, f); }, tid);
    } else {
      v_in.each([&](int r, int col, const Frag<T>& f) { VTile<T>::put(sV, r, col, f); }, tid);
    }
  };
  // state and column stores of chunk c
  const size_t chunk_state = (size_t)HV * D * D, chunk_cols = (size_t)HV * D * BT;
  C* const st_out = reinterpret_cast<C*>(back ? a.ds : a.hs) + ((size_t)j * D + vrow) * D;
  C* const col_out = reinterpret_cast<C*>(back ? a.dr : a.vn) + ((size_t)j * D + vrow) * BT;

  if (NC > 0) fetch(back ? NC - 1 : 0);
  for (int i = 0; i < NC; ++i) {
    const int c = back ? NC - 1 - i : i;
    const size_t slot = (size_t)(slot0 + c);
    __syncthreads();
    place();
    if (i + 1 < NC) fetch(back ? c - 1 : c + 1);
    __syncthreads();

    Frag<C> Sh[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      join(Sh[s], S[2 * s], S[2 * s + 1]);
      store8(st_out + slot * chunk_state + 32 * s + 8 * g, Sh[s]);
    }
    // X = K S, lane: tokens perm_row(tb, 4 g + i), column n
    f32x4 X[4];
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) X[tb] = zero4();
#pragma unroll
    for (int s = 0; s < KS; ++s)
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) X[tb] = mma(TK::row8(sK, perm_row(tb, n), 32 * s + 8 * g), Sh[s], X[tb]);
    f32x4 ex[4], ey[4], bz[4];
#pragma unroll
    for (int tb = 0; tb < 4; ++tb) {
      ex[tb] = *reinterpret_cast<const f32x4*>(sG + perm_row(tb, 4 * g));
      ey[tb] = *reinterpret_cast<const f32x4*>(sG + BT + perm_row(tb, 4 * g));
      bz[tb] = *reinterpret_cast<const f32x4*>(sG + 2 * BT + perm_row(tb, 4 * g));
    }
    const float eGl = sG[3 * BT];
    f32x4 Z[4];
    Frag<C> Zf[2];
    if (!back) {
      // R = beta (v - e^G X), Vn = A R (block lower triangular in 32-token slabs)
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) X[tb] = bz[tb] * (VTile<T>::get(sV, tb, w, n, g) - ex[tb] * X[tb]);
      Frag<C> R0, R1;
      join(R0, X[0], X[1]);
      join(R1, X[2], X[3]);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) Z[tb] = mma(TA::row8(sA, perm_row(tb, n), 8 * g), R0, zero4());
#pragma unroll
      for (int tb = 2; tb < 4; ++tb) Z[tb] = mma(TA::row8(sA, perm_row(tb, n), 32 + 8 * g), R1, Z[tb]);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        join(Zf[p], Z[2 * p], Z[2 * p + 1]);
        store8(col_out + slot * chunk_cols + 32 * p + 8 * g, Zf[p]);
        join(Zf[p], Z[2 * p] * ey[2 * p], Z[2 * p + 1] * ey[2 * p + 1]);
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) S[kb] = S[kb] * eGl;
    } else {
      // Y = e^{G_last - G} X + P^T dO, dR = A^T Y
      Frag<C> dO[2];
#pragma unroll
      for (int p = 0; p < 2; ++p) dO[p] = TA::template col8<true>(sV, 32 * p + 8 * g, w, n);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        X[tb] = X[tb] * ey[tb];
        if (tb < 2) X[tb] = mma(TA::template col8<false>(sP, 8 * g, tb, n), dO[0], X[tb]);
        X[tb] = mma(TA::template col8<false>(sP, 32 + 8 * g, tb, n), dO[1], X[tb]);
      }
      Frag<C> Y0, Y1;
      join(Y0, X[0], X[1]);
      join(Y1, X[2], X[3]);
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        Z[tb] = mma(TA::template col8<false>(sA, 32 + 8 * g, tb, n), Y1, zero4());
        if (tb < 2) Z[tb] = mma(TA::template col8<false>(sA, 8 * g, tb, n), Y0, Z[tb]);
      }
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        join(Zf[p], Z[2 * p], Z[2 * p + 1]);
        store8(col_out + slot * chunk_cols + 32 * p + 8 * g, Zf[p]);
        join(Zf[p], Z[2 * p] * (-bz[2 * p] * ex[2 * p]), Z[2 * p + 1] * (-bz[2 * p + 1] * ex[2 * p + 1]));
      }
      // dh' <- e^{G_last} dh' + Q^T (scale e^G dO)
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        f32x8 x = values(dO[p]);
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // slots 8 g + e are the tokens of blocks 2 p and 2 p + 1
          x[e] *= a.f.scale * ex[2 * p][e];
          x[4 + e] *= a.f.scale * ex[2 * p + 1][e];
        }
        join(dO[p], f32x4{x[0], x[1], x[2], x[3]}, f32x4{x[4], x[5], x[6], x[7]});
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        S[kb] = S[kb] * eGl;
#pragma unroll
        for (int p = 0; p < 2; ++p) S[kb] = mma(TK::template col8<false>(sQ, 32 * p + 8 * g, kb, n), dO[p], S[kb]);
      }
    }
    // ... + K^T Z
#pragma unroll
    for (int kb = 0; kb < KB; ++kb)
#pragma unroll
      for (int p = 0; p < 2; ++p) S[kb] = mma(TK::template col8<false>(sK, 32 * p + 8 * g, kb, n), Zf[p], S[kb]);
  }
  if (back && a.dh0) {
    T* out = reinterpret_cast<T*>(a.dh0) + sbase;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      store_io8(out + 32 * s + 8 * g, both(S[2 * s], S[2 * s + 1]) * inv);
    }
  }
}

// ---------------------------------------------------------- largest gradients
// amax[n, j] = bits of max |dht| (0 without one): one work-group a (sequence, head).
__global__ __launch_bounds__(256) void bwd_amax_init_kernel(const float* __restrict__ dht, int per,
                                                            uint32_t* __restrict__ amax) {
  __shared__ uint32_t sm[4];
  uint32_t m = 0;
  if (dht) {
    const uint4* p = reinterpret_cast<const uint4*>(dht + (size_t)blockIdx.x * per);
    for (int i = threadIdx.x; i < per / 4; i += 256) {
      const uint4 x = p[i];
      m = max(m, max(max(x.x & 0x7FFFFFFFu, x.y & 0x7FFFFFFFu), max(x.z & 0x7FFFFFFFu, x.w & 0x7FFFFFFFu)));
    }
  }
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
  __syncthreads();
  if (threadIdx.x == 0) amax[blockIdx.x] = max(max(sm[0], sm[1]), max(sm[2], sm[3]));
}

// max |dout| of 16 rows of a chunk into amax (the order does not change a maximum).
// LPH lanes hold a head's channels of a row.
template <int LPH>
__global__ __launch_bounds__(256) void bwd_amax_kernel(const bf16_t* __restrict__ dout, uint32_t* __restrict__ amax,
                                                       const int64_t* __restrict__ cu, const int32_t* __restrict__ coff,
                                                       int T, int N, int NT, int HV, int cblocks) {
  const int cb = blockIdx.x % cblocks, part = blockIdx.x / cblocks % 4, slot = blockIdx.x / cblocks / 4;
  // the chunk and its sequence
  int ns, c0, nrow;
  if (cu) {
    if (slot >= coff[N]) return;
    int lo = 0, hi = N;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (coff[mid] <= slot) lo = mid; else hi = mid;
    }
    ns = lo;
    long long b0 = cu[lo], b1 = cu[lo + 1];
    b0 = b0 < 0 ? 0 : (b0 > T ? T : b0);
    b1 = b1 < b0 ? b0 : (b1 > T ? T : b1);
    c0 = (int)b0 + 64 * (slot - coff[lo]);
    nrow = (int)b1 - c0 < 64 ? (int)b1 - c0 : 64;
  } else {
    ns = slot / NT;
    const int it = slot - ns * NT;
    c0 = ns * T + 64 * it;
    nrow = T - 64 * it < 64 ? T - 64 * it : 64;
  }
  const int ch = (cb * 256 + threadIdx.x) * 8;
  const int C = HV * LPH * 8;
  if (ch >= C) return;   // whole heads
  const int r1 = nrow < 16 * part + 16 ? nrow : 16 * part + 16;
  uint32_t m = 0;
  const bf16_t* p = dout + (size_t)c0 * C + ch;
#pragma unroll 4
  for (int r = 16 * part; r < r1; ++r) {
    const uint4 x = *reinterpret_cast<const uint4*>(p + (size_t)r * C);
    const uint32_t ws[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max(m, max((ws[i] << 16) & 0x7FFFFFFFu, ws[i] & 0x7FFF0000u));
  }
#pragma unroll
  for (int off = 1; off < LPH; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  if (threadIdx.x % LPH == 0 && m) atomicMax(amax + (size_t)ns * HV + ch / (8 * LPH), m);
}

template <typename T, int D>
hipError_t launch_scan(const ChunkBwdArgs& a, hipStream_t s) {
  typedef ScanLds<T, typename ComputeOf<T>::type, D> L;
  const long long units = ((long long)a.f.N * a.f.Hk + 7) / 8 * 8;
  const unsigned grid = (unsigned)(units * (a.f.HV / a.f.Hk) * (D / 64) * 2);
  const void* kern = reinterpret_cast<const void*>(gdn_bwd_scan_kernel<T, D>);
  if (L::bytes > 65536)
    if (hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, L::bytes)) return e;
  hipLaunchKernelGGL((gdn_bwd_scan_kernel<T, D>), dim3(grid), dim3(256), L::bytes, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk_bwd_amax(const ChunkBwdArgs& a, hipStream_t s) {
  const ChunkArgs& f = a.f;
  hipLaunchKernelGGL(bwd_amax_init_kernel, dim3((unsigned)(f.N * f.HV)), dim3(256), 0, s, a.dht, f.V * f.K, a.amax);
  if (hipError_t e = hipGetLastError()) return e;
  if ((long long)f.B * f.T == 0) return hipSuccess;
  const int cblocks = (f.HV * f.V / 8 + 255) / 256, NT = (f.T + 63) / 64;
  const dim3 grid((unsigned)((long long)a.nslots * 4 * cblocks));
  auto kern = f.V == 128 ? bwd_amax_kernel<16> : bwd_amax_kernel<8>;
  hipLaunchKernelGGL(kern, grid, dim3(256), 0, s, (const bf16_t*)a.dout, a.amax, f.cu_seqlens, f.chunk_off, f.T, f.N, NT,
                     f.HV, cblocks);
  return hipGetLastError();
}

hipError_t launch_chunk_bwd_scan(const ChunkBwdArgs& a, hipStream_t s) {
  if (a.f.bf16) return a.f.K == 128 ? launch_scan<bf16_t, 128>(a, s) : launch_scan<bf16_t, 64>(a, s);
  return a.f.K == 128 ? launch_scan<float, 128>(a, s) : launch_scan<float, 64>(a, s);
}

}  // namespace gdn
