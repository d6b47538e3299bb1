// The two sequential parts of the chunked rule's gradients, gfx950 (chunk_bwd.h
// has the mathematics): the states h and new values Vn again, first chunk to
// last, and the state gradients dh' and dR, last chunk to first.  Neither needs
// the other, and every V column of either stands for itself: one launch runs both
// at once, with twice the work-groups of one.
//
// A work-group is one (sequence, v-head, 64 columns, direction): four state waves
// of 16 columns, one per SIMD, whose state (K x 16, fp32) stays in MFMA
// accumulators, and four movers.  As in the prefill's scan, rows of the A operands
// are placed so that two accumulators are the next product's B operand, without a
// trip through LDS: K h -> R -> A R -> state, and K dh' -> Y -> A^T Y -> state.
// The movers bring the next chunk's K (and Q), A (and P), v or dO tiles into the
// other half of a double buffer in LDS, in the compute type, rows behind the
// sequence's end as zeros, with the chunk after that in flight in their registers;
// one barrier a chunk.  Row fragments are 16-byte reads; K^T, Q^T, A^T, P^T and
// dO^T come from the same tiles by transposing reads.  (fp32 tiles fit once: the
// movers then write between two barriers.)
//
// Bound by memory: 4 sequences of 4096 tokens, 16 heads of 128, bf16: 190 - 215 us, 840 MB
// at 4.2 TB/s (a large copy reaches 5.2), nearly half of it h, dh', Vn and dR on their way
// to the next launch; eight ragged sequences of 16001 tokens in all, 32 heads: 370 - 410 us,
// 1.44 GB.  With loads by the state waves themselves the first took 260 us, with stores in
// rows of the arrays instead of the order in which waves hold them the second 405.
// Where sequences x heads are few, the chunks one after the other on the few CUs that
// these fill: one sequence of 16384 tokens, 16 heads of 128, bf16: 600 us, 2.3 a chunk,
// on 64 of them.  fp32 likewise, at its products' rate: 2 x 1000 tokens, 4 heads of 64:
// 65 us, 4 us a chunk (the state gradients' five products are 288 instructions of 32
// cycles on each SIMD); the first size in fp32 917 us.
//
// h and dh' leave as [V][K], Vn and dR transposed ([V][64]): what a lane's
// accumulators hold in order, a wave's stores 1 KiB in a row.

#include "chunk_bwd.h"
#include "chunk_common.h"

namespace gdn {

namespace {

using namespace bwd;

// the sequence's bounds, clamped to the tokens
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
  static constexpr int stages = 2 * bytes <= 160 * 1024 ? 2 : 1;
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
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void gdn_bwd_scan_kernel(ChunkBwdArgs a) {
  typedef typename ComputeOf<T>::type C;
  typedef ScanLds<T, C, D> L;
  typedef Tile<C, D> TK;
  typedef Tile<C, 64> TA;
  constexpr int KS = D / 32, KB = D / 16, NVT = D / 64;
  constexpr bool TWO = L::stages == 2;
  extern __shared__ __attribute__((aligned(16))) char lds[];

  const int tid = threadIdx.x & 255, lane = tid & 63, n = lane & 15, g = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const bool mover = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8) != 0;
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
  if (back && a.amax) {
    // the largest gradient of the (sequence, key head): of dht, and of the chunks' quarters
    uint32_t* const sm = reinterpret_cast<uint32_t*>(lds);
    uint32_t m = 0;
    for (int i = threadIdx.x; i < 4 * NC * GR; i += 512) {
      const int row = i / GR;
      m = max(m, a.part[((size_t)slot0 * 4 + row) * HV + jk * GR + (i - row * GR)]);
    }
    if (a.dht)
      for (int i = threadIdx.x; i < GR; i += 512) m = max(m, a.amax_dht[(size_t)ns * HV + jk * GR + i]);
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    if (lane == 0) sm[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, sm[i]);
    __syncthreads();
    gs = grad_scale(m, inv);
    if (v0 == 0 && j == jk * GR && threadIdx.x == 0) a.amax[(size_t)ns * Hk + jk] = m;   // for the chunks' gradients
  }
  auto chunk_of = [&](int i) { return back ? NC - 1 - i : i; };

  if (mover) {
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
    auto fetch = [&](int i) {
      const int c0 = bos + BT * chunk_of(i), nrow = eos - c0 < BT ? eos - c0 : BT;
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
    auto place = [&](char* st) {
      k_in.each([&](int r, int col, const Frag<T>& f) { TK::put(st + L::K, r, col, widen(f)); }, tid);
      a_in.each([&](int r, int col, const Frag<C>& f) { TA::put(st + L::A, r, col, f); }, tid);
      reinterpret_cast<float*>(st + L::G)[tid] = gate_in;
      if (back) {
        v_in.each([&](int r, int col, const Frag<T>& f) { TA::put(st + L::V, r, col, widen(f, gs)); }, tid);
        q_in.each([&](int r, int col, const Frag<T>& f) { TK::put(st + L::Q, r, col, widen(f)); }, tid);
        p_in.each([&](int r, int col, const Frag<C>& f) { TA::put(st + L::P, r, col, f); }, tid);
      } else {
        v_in.each([&](int r, int col, const Frag<T>& f) { VTile<T>::put(st + L::V, r, col, f); }, tid);
      }
    };
    if (NC > 0) fetch(0);
    if constexpr (TWO) {
      if (NC > 0) {
        place(lds);
        if (NC > 1) fetch(1);
      }
      tiles::lds_barrier();
      for (int i = 0; i < NC; ++i) {
        if (i + 1 < NC) {
          place(lds + ((i + 1) & 1) * L::bytes);
          if (i + 2 < NC) fetch(i + 2);
        }
        tiles::lds_barrier();
      }
    } else {
      for (int i = 0; i < NC; ++i) {
        place(lds);
        if (i + 1 < NC) fetch(i + 1);
        tiles::lds_barrier();
        tiles::lds_barrier();
      }
    }
    return;
  }

  f32x4 S[KB];
  const float* init = back ? a.dht : a.f.h0;
#pragma unroll
  for (int kb = 0; kb < KB; ++kb) {
    S[kb] = zero4();
    if (init) S[kb] = *reinterpret_cast<const f32x4*>(init + sbase + perm_row(kb, 4 * g)) * gs;
  }
  // state and column stores of a chunk
  const size_t chunk_state = (size_t)HV * D * D, chunk_cols = (size_t)HV * D * BT;
  C* const st_out = reinterpret_cast<C*>(back ? a.ds : a.hs) + (size_t)j * D * D;
  C* const col_out = reinterpret_cast<C*>(back ? a.dr : a.vn) + (size_t)j * D * BT;
  const int vblk = v0 / 16 + w;

  // Keeps the order of what is issued around it: left to itself the compiler reads each
  // fragment right before its product and waits out the LDS latency every time.  (fp32
  // fragments are twice as large and do not fit that way.)
  auto fence = [&]() __attribute__((always_inline)) {
    if constexpr (sizeof(C) == 2) __builtin_amdgcn_sched_barrier(0);
  };
  // offsets of the lane's fragments in a stage
  int o_row[KS], o_k[KS];   // K (Q) rows of slab s, columns of block pair m
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    o_row[s] = TK::off(perm_row(0, n), 32 * s + 8 * g);
    o_k[s] = TK::pair_cols(s, n, g);
  }
  const int o_a[2] = {TA::off(perm_row(0, n), 8 * g), TA::off(perm_row(0, n), 32 + 8 * g)};
  const int o_at[2] = {TA::pair_cols(0, n, g), TA::pair_cols(1, n, g)};
  const int o_do = TA::block_cols(w, n, g);
  // K^T (Q^T): channels of block kb, tokens 32 p + 8 g + [0, 8); A^T, P^T alike; rows of A
  auto kt = [&](const char* t, int kb, int p) __attribute__((always_inline)) {
    return TK::col(t + o_k[kb / 2] + 32 * p * TK::pitch + (kb & 1) * TK::odd);
  };
  auto at = [&](const char* t, int tb, int p) __attribute__((always_inline)) {
    return TA::col(t + o_at[tb / 2] + 32 * p * TA::pitch + (tb & 1) * TA::odd);
  };
  auto ar = [&](const char* t, int tb, int p) __attribute__((always_inline)) {
    return TA::row(t + o_a[p] + tiles::blk_rows(tb) * TA::pitch);
  };
  if constexpr (TWO) tiles::lds_barrier();
  auto walk = [&](auto direction) __attribute__((always_inline)) {
    constexpr bool BACK = decltype(direction)::value;
    for (int i = 0; i < NC; ++i) {
      const size_t slot = (size_t)(slot0 + chunk_of(i));
      const char* const st = lds + (TWO ? (i & 1) * L::bytes : 0);
      const char* const sK = st + L::K;
      const char* const sA = st + L::A;
      const char* const sV = st + L::V;
      const float* const sG = reinterpret_cast<const float*>(st + L::G);
      const char* const sQ = st + L::Q;
      const char* const sP = st + L::P;
      if constexpr (!TWO) tiles::lds_barrier();

      // lane: tokens perm_row(tb, 4 g + i), column n
      f32x4 X[4], Z[4], ex[4], ey[4], bz[4], v[4];
      Frag<C> Kr[KS][4], Ar[6], Pt[6], Sh[KS], Zf[2], dO[2], Q0[KB], Q1[KB], K0[KB], K1[KB];
      // ---- what the first products need
      auto gates = [&](f32x4 (&x)[4], int plane) __attribute__((always_inline)) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) x[tb] = *reinterpret_cast<const f32x4*>(sG + plane * BT + perm_row(tb, 4 * g));
      };
      const float eGl = sG[3 * BT];
      if constexpr (BACK) {
#pragma unroll
        for (int p = 0; p < 2; ++p) dO[p] = TA::col(sV + o_do + 32 * p * TA::pitch);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) Pt[tb] = at(sP, tb, 1);
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) Pt[4 + tb] = at(sP, tb, 0);
      } else {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) v[tb] = VTile<T>::get(sV, tb, w, n, g);
      }
      auto k_rows = [&](int s) __attribute__((always_inline)) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) Kr[s][tb] = TK::row(sK + o_row[s] + tiles::blk_rows(tb) * TK::pitch);
      };
#pragma unroll
      for (int s = 0; s < KS / 2; ++s) k_rows(s);
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        join(Sh[s], S[2 * s], S[2 * s + 1]);
        store8(st_out + slot * chunk_state + Kept<C, D>::at(vblk, s, n, g), Sh[s]);
      }
      fence();
      // ---- P^T dO and X = K S; meanwhile the rows of A (A^T), then Q^T or K^T
      if constexpr (BACK) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) Z[tb] = mma(Pt[tb], dO[1], zero4());
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) Z[tb] = mma(Pt[4 + tb], dO[0], Z[tb]);
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) X[tb] = zero4();
#pragma unroll
      for (int s = 0; s < KS; ++s) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) X[tb] = mma(Kr[s][tb], Sh[s], X[tb]);
        if (s < KS / 2) k_rows(s + KS / 2);
        if (s == KS / 2 - 1) {
#pragma unroll
          for (int tb = 0; tb < 4; ++tb) Ar[tb] = BACK ? at(sA, tb, 1) : ar(sA, tb, 0);
#pragma unroll
          for (int tb = 0; tb < 2; ++tb) Ar[4 + tb] = BACK ? at(sA, tb, 0) : ar(sA, 2 + tb, 1);
        }
        if (s == KS - 1) {
          gates(ex, 0);
          if constexpr (BACK) gates(ey, 1);
          else gates(bz, 2);
#pragma unroll
          for (int kb = 0; kb < KB; ++kb) (BACK ? Q0 : K0)[kb] = kt(BACK ? sQ : sK, kb, 0);
        }
        fence();
      }
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) S[kb] = S[kb] * eGl;
      if constexpr (!BACK) {
        // R = beta (v - e^G X), Vn = A R (block lower triangular in 32-token slabs)
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) X[tb] = bz[tb] * (v[tb] - ex[tb] * X[tb]);
        Frag<C> R0, R1;
        join(R0, X[0], X[1]);
        join(R1, X[2], X[3]);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) Z[tb] = mma(Ar[tb], R0, zero4());
#pragma unroll
        for (int tb = 2; tb < 4; ++tb) Z[tb] = mma(Ar[2 + tb], R1, Z[tb]);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) K1[kb] = kt(sK, kb, 1);
        gates(ey, 1);
        fence();
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          join(Zf[p], Z[2 * p], Z[2 * p + 1]);
          store8(col_out + slot * chunk_cols + Kept<C, 64>::at(vblk, p, n, g), Zf[p]);
          join(Zf[p], Z[2 * p] * ey[2 * p], Z[2 * p + 1] * ey[2 * p + 1]);
        }
      } else {
        // dh' <- e^{G_last} dh' + Q^T (scale e^G dO), which waits for nothing; Y =
        // e^{G_last - G} X + P^T dO, dR = A^T Y
#pragma unroll
        for (int p = 0; p < 2; ++p) {   // slots 8 g + e are the tokens of blocks 2 p and 2 p + 1
          const f32x8 x = values(dO[p]);
          join(dO[p], f32x4{x[0], x[1], x[2], x[3]} * (ex[2 * p] * a.f.scale),
               f32x4{x[4], x[5], x[6], x[7]} * (ex[2 * p + 1] * a.f.scale));
        }
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) Q1[kb] = kt(sQ, kb, 1);
        fence();
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) S[kb] = mma(Q0[kb], dO[0], S[kb]);
        Frag<C> Y0, Y1;
        join(Y0, X[0] * ey[0] + Z[0], X[1] * ey[1] + Z[1]);
        join(Y1, X[2] * ey[2] + Z[2], X[3] * ey[3] + Z[3]);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) K0[kb] = kt(sK, kb, 0);
        gates(bz, 2);
        fence();
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) Z[tb] = mma(Ar[tb], Y1, zero4());
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) Z[tb] = mma(Ar[4 + tb], Y0, Z[tb]);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) S[kb] = mma(Q1[kb], dO[1], S[kb]);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) K1[kb] = kt(sK, kb, 1);
        fence();
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          join(Zf[p], Z[2 * p], Z[2 * p + 1]);
          store8(col_out + slot * chunk_cols + Kept<C, 64>::at(vblk, p, n, g), Zf[p]);
          join(Zf[p], Z[2 * p] * (-bz[2 * p] * ex[2 * p]), Z[2 * p + 1] * (-bz[2 * p + 1] * ex[2 * p + 1]));
        }
      }
      // ... + K^T Z
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) S[kb] = mma(K0[kb], Zf[0], S[kb]);
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) S[kb] = mma(K1[kb], Zf[1], S[kb]);
      tiles::lds_barrier();
    }
  };
  if (back) walk(tiles::Stage1{});
  else walk(tiles::Stage0{});
  if (back && a.dh0) {
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const f32x8 x = both(S[2 * s], S[2 * s + 1]) * inv;
      const size_t at = sbase + 32 * s + 8 * g;
      if (a.f32) store_io8(reinterpret_cast<float*>(a.dh0) + at, x);
      else store_io8(reinterpret_cast<T*>(a.dh0) + at, x);
    }
  }
}

// ---------------------------------------------------------- largest gradients
// part[slot][quarter][head] = bits of max |dout| of 16 rows of a chunk, LPH lanes a head's
// channels of a row; the last `states` work-groups: amax_dht[n, j] = bits of max |dht|.
// Every maximum has a place of its own, which the scans read: no atomics, nothing to
// clear.  A read of dout: 67 MB in 16 us, 131 MB in 30 us (4.3 TB/s).
template <int LPH>
__global__ __launch_bounds__(256) void bwd_amax_kernel(ChunkBwdArgs a, int cblocks, int states) {
  __shared__ uint32_t sm[4];
  uint32_t m = 0;
  const int first = (int)gridDim.x - states;
  if ((int)blockIdx.x >= first) {
    const int cell = (int)blockIdx.x - first, per = a.f.V * a.f.K;
    const uint4* p = reinterpret_cast<const uint4*>(a.dht + (size_t)cell * per);
    for (int i = threadIdx.x; i < per / 4; i += 256) {
      const uint4 x = p[i];
      m = max(m, max(max(x.x & 0x7FFFFFFFu, x.y & 0x7FFFFFFFu), max(x.z & 0x7FFFFFFFu, x.w & 0x7FFFFFFFu)));
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
    if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) a.amax_dht[cell] = max(max(sm[0], sm[1]), max(sm[2], sm[3]));
    return;
  }
  const int cb = blockIdx.x % cblocks, part = blockIdx.x / cblocks % 4, slot = blockIdx.x / cblocks / 4;
  int c0, nrow;
  if (!intra::locate_chunk(slot, a.f.cu_seqlens, a.f.chunk_off, a.f.N, a.f.T, (a.f.T + BT - 1) / BT, c0, nrow)) return;
  const int ch = (cb * 256 + threadIdx.x) * 8;
  const int HV = a.f.HV, C = HV * LPH * 8;
  if (ch >= C) return;   // whole heads
  const bf16_t* p = reinterpret_cast<const bf16_t*>(a.dout) + (size_t)c0 * C + ch;
  uint4 x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {   // rows behind the end: the last one again
    const int r = 16 * part + i < nrow ? 16 * part + i : nrow - 1;
    x[i] = *reinterpret_cast<const uint4*>(p + (size_t)r * C);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t ws[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) m = max(m, max((ws[e] << 16) & 0x7FFFFFFFu, ws[e] & 0x7FFF0000u));
  }
#pragma unroll
  for (int off = 1; off < LPH; off <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, off, 64));
  if (threadIdx.x % LPH == 0) a.part[((size_t)slot * 4 + part) * HV + ch / (8 * LPH)] = m;
}

template <typename T, int D>
hipError_t launch_scan(const ChunkBwdArgs& a, hipStream_t s) {
  typedef ScanLds<T, typename ComputeOf<T>::type, D> L;
  const long long units = ((long long)a.f.N * a.f.Hk + 7) / 8 * 8;
  const unsigned grid = (unsigned)(units * (a.f.HV / a.f.Hk) * (D / 64) * 2);
  const void* kern = reinterpret_cast<const void*>(gdn_bwd_scan_kernel<T, D>);
  const int bytes = L::stages * L::bytes;
  if (bytes > 65536)
    if (hipError_t e = hipFuncSetAttribute(kern, hipFuncAttributeMaxDynamicSharedMemorySize, bytes)) return e;
  hipLaunchKernelGGL((gdn_bwd_scan_kernel<T, D>), dim3(grid), dim3(512), bytes, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk_bwd_amax(const ChunkBwdArgs& a, hipStream_t s) {
  const ChunkArgs& f = a.f;
  const int cblocks = (f.HV * f.V / 8 + 255) / 256, states = a.dht ? f.N * f.HV : 0;
  const long long chunks = (long long)f.B * f.T > 0 ? (long long)a.nslots * 4 * cblocks : 0;
  if (chunks + states == 0) return hipSuccess;
  const dim3 grid((unsigned)(chunks + states));
  if (f.V == 128) hipLaunchKernelGGL((bwd_amax_kernel<16>), grid, dim3(256), 0, s, a, cblocks, states);
  else hipLaunchKernelGGL((bwd_amax_kernel<8>), grid, dim3(256), 0, s, a, cblocks, states);
  return hipGetLastError();
}

hipError_t launch_chunk_bwd_scan(const ChunkBwdArgs& a, hipStream_t s) {
  if (a.f.bf16) return a.f.K == 128 ? launch_scan<bf16_t, 128>(a, s) : launch_scan<bf16_t, 64>(a, s);
  return a.f.K == 128 ? launch_scan<float, 128>(a, s) : launch_scan<float, 64>(a, s);
}

}  // namespace gdn
