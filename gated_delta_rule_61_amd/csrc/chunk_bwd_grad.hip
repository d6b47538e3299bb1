// The chunk-parallel part of the chunked rule's gradients, gfx950 (chunk_bwd.h has
// the mathematics): dq, dk, dv, dg and dbeta of a chunk from the states, the state
// gradients, Vn and dR that the two scans left.
//
// A work-group is one (chunk, key head): it takes the v-heads that share the key
// head in turn, in order, and their dq and dk add up where they are made: the rows
// of dO, dR and Vn enter the products times their tokens' gate factors, so that the
// accumulators need none (a head's share of q . dq and k . dk is what they grew by).  Products run
// transposed ([K channels] x [tokens]), so that a lane ends with 8 consecutive
// channels of a token: 16-byte stores, and the dot products with q and k (which
// make dg and dbeta) in registers.  Each of the eight waves has 32 channels of some
// token blocks; reductions over V go in blocks of 32 columns, whose tiles (Vn, dR,
// h, dh' straight to LDS, dO through registers, scaled on its way) fill one half of
// a double buffer while the other is used: one barrier a block.  The scores dO Vn^T
// and dR Vn^T are dealt out to the waves in 16 x 16 blocks, gated and masked there
// and shared through LDS, in the bytes of the tiles that are no longer needed.
//
// Bound by memory: 4 sequences of 4096 tokens, 16 heads of 128, bf16: 183 - 196 us, 911 MB
// at 4.8 TB/s; eight ragged sequences of 16001 tokens in all, 16 x 32 heads: 330 - 350 us.
// 128 registers, so that two work-groups share a CU and one's loads cover the other's
// products; with a work-group a v-head the second size took 510 us.  Two chunks of two
// heads of 128: 24 us, the latency of eight blocks, one after the other.

#include "chunk_bwd.h"
#include "chunk_common.h"

namespace gdn {

namespace {

using namespace bwd;

constexpr int NTHREADS = 512;
constexpr int VC = 32;   // V columns of a block

// A stage holds a block's Vn^T and dR^T [v][t], h and dh' [v][k], and dO [t][v].  Later
// the scores lie in the first stage, k and q [t][channel] in the second.
template <typename C, int D>
struct GradLds {
  typedef Tile<C, 64> T64;
  typedef Tile<C, D> TD;
  // dO rows: 64 bytes of fp16 (a fragment read takes 1 KiB in a row), fp32 padded
  static constexpr int orow = sizeof(C) == 2 ? 64 : 4 * VC + 16;
  static constexpr int VN = 0, DR = Kept<C, 64>::bytes, H = 2 * DR, DS = H + Kept<C, D>::bytes, O = DS + Kept<C, D>::bytes;
  static constexpr int tiles = O + BT * orow;
  static constexpr int S1 = 0, S2 = T64::bytes(BT), S3 = 2 * S2, scores = 3 * S2;
  static constexpr int K = 0, Q = TD::bytes(BT), rows = 2 * Q;
  static constexpr int more(int a, int b) { return a > b ? a : b; }
  static constexpr int first = more(tiles, scores), second = more(tiles, rows);
};

// `bytes` behind a uniform address: one 32-bit register for the lane
template <typename T>
__device__ __forceinline__ const T* ahead(const T* p, uint32_t bytes) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + bytes);
}
template <typename T>
__device__ __forceinline__ T* ahead(T* p, uint32_t bytes) {
  return reinterpret_cast<T*>(reinterpret_cast<char*>(p) + bytes);
}

// The copies of a block's four tiles on their way: straight to LDS, as they are (fp16), or
// through registers (fp32).
template <typename C, int D> struct BlockIn;
template <int D> struct BlockIn<f16_t, D> {
  typedef GradLds<f16_t, D> L;
  static constexpr int N64 = VC * 64 * 2 / 1024, ND = VC * D * 2 / 1024;   // 1 KiB pieces of a tile
  uint32_t from;
  __device__ __forceinline__ void init(int, int lane) { from = 16 * lane; }
  __device__ __forceinline__ void issue(const f16_t* vn, const f16_t* dr, const f16_t* h, const f16_t* ds, char* st, int w) {
    typedef __attribute__((address_space(3))) char lchar;
    const uint32_t at = opaque(from);
#pragma unroll
    for (int i = 0; i < (2 * N64 + 2 * ND) / 8; ++i) {
      const int p = w + 8 * i;   // uniform
      const bool cols = p < 2 * N64;
      const int q = cols ? p : p - 2 * N64, per = cols ? N64 : ND, piece = q % per * 1024;
      const f16_t* src = cols ? (q < per ? vn : dr) : (q < per ? h : ds);
      const int to = cols ? (q < per ? L::VN : L::DR) : (q < per ? L::H : L::DS);
      tiles::dma16(ahead(reinterpret_cast<const char*>(src) + piece, at), (lchar*)(st + to + piece));
    }
  }
  __device__ __forceinline__ void commit(char*, int) { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
};
template <int D> struct BlockIn<float, D> {
  typedef GradLds<float, D> L;
  static constexpr int NW = VC * D / 8 / (NTHREADS / 2);   // vectors of h or dh' for each half of the threads
  Frag<float> cols, wide[NW];
  int t;
  __device__ __forceinline__ void init(int w, int lane) { t = (w & 3) * 64 + lane; }
  __device__ __forceinline__ void issue(const float* vn, const float* dr, const float* h, const float* ds, char*, int w) {
    load8(cols, (w < 4 ? vn : dr) + t * 8);
#pragma unroll
    for (int i = 0; i < NW; ++i) load8(wide[i], (w < 4 ? h : ds) + (t + 256 * i) * 8);
  }
  __device__ __forceinline__ void commit(char* st, int tid) {
    const bool first = tid < 256;
    Tile<float, 64>::put(st + (first ? L::VN : L::DR), t / 8, t % 8 * 8, cols);
#pragma unroll
    for (int i = 0; i < NW; ++i) {
      const int v = t + 256 * i;
      Tile<float, D>::put(st + (first ? L::H : L::DS), v / (D / 8), v % (D / 8) * 8, wide[i]);
    }
  }
};

template <typename T, int D>
__global__ __launch_bounds__(NTHREADS) __attribute__((amdgpu_waves_per_eu(sizeof(T) == 2 ? 4 : 2))) void gdn_bwd_grad_kernel(
    ChunkBwdArgs a) {
  typedef typename ComputeOf<T>::type C;
  typedef GradLds<C, D> L;
  typedef Tile<C, D> TD;
  typedef Tile<C, 64> T64;
  typedef Kept<C, D> KD;
  typedef Kept<C, 64> K64;
  constexpr int VB = D / VC;          // blocks of V columns (an even number)
  constexpr int KW = D / 32;          // waves side by side over the channels
  constexpr int NT = KW / 2;          // 16-token blocks of a wave
  __shared__ __attribute__((aligned(16))) char st0[L::first], st1[L::second];
  // G, e^G, e^{G_last - G}, beta of the tokens; dot products, one row for 32 channels;
  // v . dR; <h, dh'> of each wave
  __shared__ __attribute__((aligned(16))) float sG[4 * BT], red[16 * BT], sVdr[2 * BT], sHd[8];
  // q . dq and k . dk (the lane's channels) of the heads so far
  __shared__ float sDone[2 * NT][NTHREADS];

  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = w % KW, th = w / KW, tb0 = th * NT;   // the wave's channels 32 kw .. and token blocks
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

  f32x4 dq[2][NT], dk[2][NT];   // sums over the heads
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) dq[h][t] = dk[h][t] = zero4();
  // every gradient of the key head's v-heads is kept times one power of two
  float inv = 1.f, gs = 1.f;
  if (a.amax) gs = grad_scale(a.amax[(size_t)ns * Hk + jk], inv);
  // the wave's block of the scores: lower blocks (tb, sb) in the order of tix
  const int tbw = w >= 6 ? 3 : w >= 3 ? 2 : w >= 1 ? 1 : 0, sbw = w - tbw * (tbw + 1) / 2;
  Frag<T> o_in, v_in;   // dO and v of the block on its way
  for (int r = 0; r < GR; ++r) {
    // what a lane derives from its place it derives once a head (see opaque)
    const int tid = opaque((int)threadIdx.x), lane = tid & 63, n = lane & 15, g = lane >> 4;
    // where the lane's fragments lie in a tile
    const int pair0 = KD::pair_cols(kw, n, g);       // channels 32 kw .., 8 rows
    const int block0 = K64::block_cols(n, g);        // 16 tokens, 8 rows
    const int row0 = n * L::orow + 8 * g * (int)sizeof(C);
    // the rows of dO that this thread brings (the first 256), the token and columns whose v it meets
    const int ot = tid / 4 & 63, oc = tid % 4 * 8;
    const int vt = 16 * (w & 3) + n;
    // byte offsets of this thread's rows behind uniform addresses (64 rows: below 2^32)
    const uint32_t o_off = ((uint32_t)(ot < nrow ? ot : nrow - 1) * (uint32_t)vstride + oc) * sizeof(T);
    const uint32_t v_off = ((uint32_t)(vt < nrow ? vt : nrow - 1) * (uint32_t)vstride + 8 * g) * sizeof(T);
    BlockIn<C, D> in;
    in.init(w, lane);
    const int j = jk * GR + r;
    T* const dvp = reinterpret_cast<T*>(a.dv) + (size_t)c0 * vstride + (size_t)j * D;

    Frag<T> k_in[D / 64], q_in[D / 64];
    auto issue = [&](int vb, char* st) __attribute__((always_inline)) {
      const size_t cell = (size_t)slot * HV + j, first = (size_t)c0 * vstride + (size_t)j * D + VC * vb;
      if (tid < 256) load8(o_in, ahead(reinterpret_cast<const T*>(a.dout) + first, opaque(o_off)));
      if ((vb & 1) == w >> 2) load8(v_in, ahead(reinterpret_cast<const T*>(a.f.v) + first, opaque(v_off)));
      in.issue(reinterpret_cast<const C*>(a.vn) + (cell * D + VC * vb) * BT,
               reinterpret_cast<const C*>(a.dr) + (cell * D + VC * vb) * BT,
               reinterpret_cast<const C*>(a.hs) + (cell * D + VC * vb) * D,
               reinterpret_cast<const C*>(a.ds) + (cell * D + VC * vb) * D, st, w);
    };
    auto fetch_rows = [&](int tid) __attribute__((always_inline)) {   // k and q for the products within the chunk
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int x = tid + NTHREADS * i, t = x / (D / 8), c = x % (D / 8) * 8;
        const uint32_t off = ((uint32_t)(t < nrow ? t : nrow - 1) * (uint32_t)krow + c) * sizeof(T);
        load8(k_in[i], ahead(kp, off));
        load8(q_in[i], ahead(qp, off));
      }
    };
    auto put_rows = [&](int tid, char* sK, char* sQ) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < D / 64; ++i) {
        const int x = tid + NTHREADS * i, t = x / (D / 8), c = x % (D / 8) * 8;
        Frag<C> kk = widen(k_in[i]), qq = widen(q_in[i]);
        if (t >= nrow) {
          kk.zero();
          qq.zero();
        }
        TD::put(sK, t, c, kk);
        TD::put(sQ, t, c, qq);
      }
    };
    auto commit = [&](char* st) __attribute__((always_inline)) {
      in.commit(st, tid);
      if (tid < 256) {
        Frag<C> f = widen(o_in, gs);
        if (ot >= nrow) f.zero();
        if constexpr (sizeof(C) == 2) *reinterpret_cast<f16x8*>(st + L::O + ot * L::orow + 2 * oc) = f.v;
        else *reinterpret_cast<f32x8*>(st + L::O + ot * L::orow + 4 * oc) = f.v;
      }
    };
    issue(0, st0);
    // the gates: G again from its terms, beta
    if (w == 7) {
      const int tl = lane < nrow ? lane : nrow - 1;
      const float graw = a.f.g ? a.f.g[(size_t)(c0 + tl) * HV + j] : (a.f.g_gamma ? a.f.g_gamma[j] : 0.f);
      const float b = a.f.beta[(size_t)(c0 + tl) * HV + j];
      const float G = intra::wave_incl_scan(lane < nrow ? intra::log_gate(graw) : 0.f, lane);
      const float Gl = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, G), nrow - 1));
      sG[lane] = G;
      sG[BT + lane] = __expf(G);
      sG[2 * BT + lane] = lane < nrow ? __expf(Gl - G) : 0.f;
      sG[3 * BT + lane] = lane < nrow ? b : 0.f;
    }

    f32x4 E[2][NT], M[3];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int t = 0; t < NT; ++t) E[h][t] = zero4();
#pragma unroll
    for (int i = 0; i < 3; ++i) M[i] = zero4();
    float hd = 0.f;        // <h, dh'>, the lane's elements
    float vdr = 0.f;       // v . dR of token vt, the lane's columns
    auto step = [&](int vb, char* st, char* next) __attribute__((always_inline)) {
      commit(st);
      tiles::lds_barrier();
      const int o_pair = opaque(pair0), o_block = opaque(block0), o_row = opaque(row0);
      // dv of token vt, and v . dR (a transposing read takes part of its addresses from
      // other lanes: all of them, also behind the end, where dR is 0)
      if ((vb & 1) == w >> 2) {
        const f32x8 x = values(K64::col(st + L::DR, K64::to_block(o_block, w & 3))), y = values(v_in);
#pragma unroll
        for (int e = 0; e < 8; ++e) vdr = fmaf(x[e], y[e], vdr);
        if (vt < nrow) store_io8(ahead(dvp + VC * vb, opaque(v_off)), x * (sG[3 * BT + vt] * inv));
      }
      if (vb + 1 < VB) issue(vb + 1, next);
      Frag<C> hf[2], df[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        hf[h] = KD::col(st + L::H + h * KD::odd, o_pair);
        df[h] = KD::col(st + L::DS + h * KD::odd, o_pair);
      }
      // each pair of waves with the same channels takes one half of <h, dh'>
      if (th < 2) {
        const f32x8 x = values(th ? hf[1] : hf[0]), y = values(th ? df[1] : df[0]);
#pragma unroll
        for (int e = 0; e < 8; ++e) hd = fmaf(x[e], y[e], hd);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tb = tb0 + t;
        // with their tokens' factors: the accumulators go on from head to head
        const float ex = sG[BT + 16 * tb + n], ey = sG[2 * BT + 16 * tb + n];
        const Frag<C> of = times(T64::row(st + L::O + 16 * tb * L::orow + o_row), a.f.scale * ex);
        const Frag<C> rf = times(K64::col(st + L::DR, K64::to_block(o_block, tb)), -ex);
        const Frag<C> vf = times(K64::col(st + L::VN, K64::to_block(o_block, tb)), ey);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          dq[h][t] = mma(hf[h], of, dq[h][t]);
          E[h][t] = mma(hf[h], rf, E[h][t]);
          dk[h][t] = mma(df[h], vf, dk[h][t]);
        }
      }
      // scores, transposed: blocks `w` (and 8 + w % 2, dealt to four waves) of both
      const Frag<C> vf = K64::col(st + L::VN, K64::to_block(o_block, sbw));
      M[0] = mma(vf, T64::row(st + L::O + 16 * tbw * L::orow + o_row), M[0]);
      M[1] = mma(vf, K64::col(st + L::DR, K64::to_block(o_block, tbw)), M[1]);
      if (w < 4) {
        const Frag<C> vl = K64::col(st + L::VN, K64::to_block(o_block, 2 + (w & 1)));
        M[2] = mma(vl, w < 2 ? T64::row(st + L::O + 48 * L::orow + o_row)
                             : K64::col(st + L::DR, K64::to_block(o_block, 3)), M[2]);
      }
    };
#pragma unroll 1
    for (int vb = 0; vb < VB; vb += 2) {
      step(vb, st0, st1);
      step(vb + 1, st1, st0);
    }

    {
      // the lane's place once more: what is derived from it stays out of the blocks' registers
      const int tid = opaque((int)threadIdx.x), lane = tid & 63, n = lane & 15, g = lane >> 4;
      const int vt = 16 * (w & 3) + n;
      fetch_rows(tid);
      // the scores, in the bytes of the first stage, whose last readers have passed a barrier
      char* const S1 = st0 + L::S1;    // scale dO Vn^T o Gamma, s <= t
      char* const S2 = st0 + L::S2;    // -dR Vn^T o Gamma, s < t
      char* const S3 = st0 + L::S3;    // beta_t times that
      auto put_score = [&](const f32x4& m, bool second, int tb, int sb) __attribute__((always_inline)) {
        const int t = 16 * tb + n, s = 16 * sb + 4 * g;
        const float Gt = sG[t], f = second ? -1.f : a.f.scale;
        const f32x4 Gs = *reinterpret_cast<const f32x4*>(sG + s);
        f32x4 x;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const bool keep = second ? s + e < t : s + e <= t;
          x[e] = keep ? f * m[e] * __expf(Gt - Gs[e]) : 0.f;
        }
        T64::put4(second ? S2 : S1, t, s, x);
        if (second) T64::put4(S3, t, s, x * sG[3 * BT + t]);
      };
      put_score(M[0], false, tbw, sbw);
      put_score(M[1], true, tbw, sbw);
      if (w < 2) put_score(M[2], false, 3, 2 + w);
      else if (w < 4) put_score(M[2], true, 3, w);
      // the blocks above the diagonal that a 32-wide slab takes in
      if (w < 6) {
        const float z = opaque(0.f);
        char* const tile = w / 2 == 0 ? S1 : w / 2 == 1 ? S2 : S3;
        T64::put4(tile, 32 * (w & 1) + n, 32 * (w & 1) + 16 + 4 * g, f32x4{z, z, z, z});
      }
      tiles::lds_barrier();
      char* const sK = st1 + L::K;
      char* const sQ = st1 + L::Q;
      put_rows(tid, sK, sQ);
      tiles::lds_barrier();

      const int o_pair = opaque(TD::pair_cols(kw, n, g)), o_block = opaque(T64::block_cols(0, n, g));
      const int o_score = opaque(T64::off(n, 8 * g)), o_chan = opaque(TD::off(n, 32 * kw + 8 * g));
      // the dot product with k of what crosses the chunk's end
      float wi[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const f32x8 k8 = values(TD::row(sK + TD::to_rows(o_chan, tb0 + t)));
        wi[t] = r == 0 ? 0.f : -sDone[NT + t][threadIdx.x];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) wi[t] = fmaf(k8[4 * h + e], dk[h][t][e], wi[t]);
      }
      // products within the chunk: only slabs that meet entries below the diagonal
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        Frag<C> ka[2], qa[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ka[h] = TD::col(sK + o_pair + 32 * p * TD::pitch + h * TD::odd);
          qa[h] = TD::col(sQ + o_pair + 32 * p * TD::pitch + h * TD::odd);
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const int tb = tb0 + t;
          if (2 * p <= tb) {   // s of the slab up to t
            const int at = T64::to_rows(o_score, tb, p);
            const Frag<C> s1 = T64::row(S1 + at), s2 = T64::row(S2 + at);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              dq[h][t] = mma(ka[h], s1, dq[h][t]);
              E[h][t] = mma(ka[h], s2, E[h][t]);
            }
          }
          if (2 * p + 1 >= tb) {   // t of the slab from s = 16 tb + n on
            const int at = T64::to_block(o_block, tb) + 32 * p * T64::pitch;
            const Frag<C> s1 = T64::col(S1 + at), s3 = T64::col(S3 + at);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              dk[h][t] = mma(qa[h], s1, dk[h][t]);
              dk[h][t] = mma(ka[h], s3, dk[h][t]);
            }
          }
        }
      }
      // dots over the wave's channels (k and q read again: registers)
      const int o_again = opaque(o_chan);
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int tok = 16 * (tb0 + t) + n, at = TD::to_rows(o_again, tb0 + t);
        const f32x8 k8 = values(TD::row(sK + at)), q8 = values(TD::row(sQ + at));
        // q . dq, k . E, k . W and the part of k . W that crosses the end, of this head
        float before_q = 0.f, before_k = 0.f;
        if (r > 0) {
          before_q = sDone[t][threadIdx.x];
          before_k = sDone[NT + t][threadIdx.x];
        }
        float d[4] = {-before_q, 0.f, -before_k, wi[t]};
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            d[0] = fmaf(q8[4 * h + e], dq[h][t][e], d[0]);
            d[1] = fmaf(k8[4 * h + e], E[h][t][e], d[1]);
            d[2] = fmaf(k8[4 * h + e], dk[h][t][e], d[2]);
          }
        // dk = beta E + W
        const float b = sG[3 * BT + tok];
        if (r + 1 < GR) {
          sDone[t][threadIdx.x] = before_q + d[0];
          sDone[NT + t][threadIdx.x] = before_k + fmaf(b, d[1], d[2]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) dk[h][t] += E[h][t] * b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          d[i] += __shfl_xor(d[i], 16, 64);
          d[i] += __shfl_xor(d[i], 32, 64);
          if (g == 0) red[(i * 4 + kw) * BT + tok] = d[i];
        }
      }
      vdr += __shfl_xor(vdr, 16, 64);
      vdr += __shfl_xor(vdr, 32, 64);
      if (g == 0) sVdr[(w >> 2) * BT + vt] = vdr;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) hd += __shfl_xor(hd, off, 64);
      if (lane == 0) sHd[w] = hd;
      tiles::lds_barrier();
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
        float hh = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c) hh += sHd[c];
        cross += sG[BT + nrow - 1] * hh;
        // sums from each row to the end
#pragma unroll
        for (int off = 1; off < 64; off <<= 1) {
          const float y = __shfl_down(dG, off, 64);
          if (lane + off < 64) dG += y;
        }
        if (live) {
          const size_t at = (size_t)(c0 + lane) * HV + j;
          const float dg = (dG + cross) * inv, db = (sVdr[lane] + sVdr[BT + lane] + d[1]) * inv;
          if (a.f32) {
            if (a.dg) reinterpret_cast<float*>(a.dg)[at] = dg;
            reinterpret_cast<float*>(a.dbeta)[at] = db;
          } else {
            if (a.dg) reinterpret_cast<T*>(a.dg)[at] = from_f<T>(dg);
            reinterpret_cast<T*>(a.dbeta)[at] = from_f<T>(db);
          }
        }
      }
    }
    if (r + 1 < GR) tiles::lds_barrier();   // the tiles, gates and dots are written again for the next head
  }
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int tok = 16 * (tb0 + t) + n;
    if (tok < nrow) {
      const size_t at = (size_t)(c0 + tok) * krow + (size_t)jk * D + 32 * kw + 8 * g;
      store_io8(reinterpret_cast<T*>(a.dq) + at, both(dq[0][t], dq[1][t]) * inv);
      store_io8(reinterpret_cast<T*>(a.dk) + at, both(dk[0][t], dk[1][t]) * inv);
    }
  }
}

template <typename T, int D>
hipError_t launch_grad(const ChunkBwdArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((gdn_bwd_grad_kernel<T, D>), dim3(intra::intra_blocks(a.nslots, a.f.Hk)), dim3(NTHREADS), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_chunk_bwd_grad(const ChunkBwdArgs& a, hipStream_t s) {
  if (a.f.bf16) return a.f.K == 128 ? launch_grad<bf16_t, 128>(a, s) : launch_grad<bf16_t, 64>(a, s);
  return a.f.K == 128 ? launch_grad<float, 128>(a, s) : launch_grad<float, 64>(a, s);
}

}  // namespace gdn
