// Selective state-space scan for prompts, gfx950.  Per sequence and head, with
// D_t = softplus(dt_t + dt_bias) and a_t = exp(-exp(A_log) D_t),
//
//   S_t = a_t S_{t-1} + D_t x_t B_t^T,    y_t = (S_t C_t + D x_t) silu(z_t),
//
// S [V, K] (K contiguous), B and C shared by HV / Hk heads.  Over a chunk of 64
// tokens, with G_t the sum of log2 a over the chunk's tokens up to t and S the
// state before it,
//
//   Y^T = 2^{G_t} (S C^T)        + x^T M^T,  M_ts = 2^{G_t - G_s} D_s (C_t . B_s), s <= t
//   S  <- 2^{G_63} S             + sum_s (D_s 2^{G_63 - G_s} x_s) B_s^T
//
// so the work is four products of 64 x {64, K} tiles per head (one, C B^T, is
// shared by the two heads of a work-group), on the bf16 matrix cores for bf16 io
// and the fp32 ones for fp32 io.
//
// Work is cut into (sequence segment, 64 or 128 value columns).  A work-group of
// four waves walks the chunks of its segment with the state in accumulators:
// wave w owns 16 or 32 columns and all K channels, so S^T feeds both products
// from registers, and only the 64 x 64 matrix M passes through LDS.  The next
// chunk's tiles are loaded into registers while this one computes.  Where
// sequences x heads are too few for the chip, sequences are split: a first
// launch computes each segment's own final state (from zeros) and log-decay,
// and the segment's work-group of the second launch starts from the decayed sum
// of those before it (and h0).  That reads x and B twice but moves no
// per-chunk states.
//
// Precision.  Gate sums are taken in 64 bits and used as an fp32 pair, so that a
// difference G_t - G_s keeps its last places however strong the decay before it.
// A state that leaves the kernel (ht, and a segment's state handed on) is formed
// from the exact products of B with the scaled x as three bf16 terms (24 bits);
// the state that only feeds this segment's bf16 y takes one term, and S and M
// are rounded to bf16 as operands.

#include "gdn_device.h"
#include "mixer_launch.h"
#include "scan_tiles.h"

namespace gdn {

namespace {

using tiles::BT;
using tiles::perm_row;
using tiles::u32x4;

constexpr int NT = 256;   // four waves

// ------------------------------------------------------------ LDS tiles
// A tile of 64 rows (tokens) by COLS.  bf16: 16-byte units swizzled by row
// (scan_tiles.h: both row fragments and transposing reads are conflict-free);
// fp32: rows padded by one 16-byte unit.
template <typename T, int COLS> struct Tile;
template <int COLS> struct Tile<bf16_t, COLS> {
  static constexpr int bytes = BT * COLS * 2;
  static constexpr int units = COLS / 8;   // 16-byte units of a row
  static __device__ __forceinline__ int off(int row, int u) { return tiles::qk_off<COLS>(row, u); }
  // slots 32 slab + 8 q + e of a row
  static __device__ __forceinline__ Frag<bf16_t> row_frag(const char* t, int row, int slab, int q) {
    Frag<bf16_t> f;
    f.v = *reinterpret_cast<const bf16x8*>(t + off(row, 4 * slab + q));
    return f;
  }
  // column `col(c)` + r % 4 of chunk c = r / 4 at tokens s0 + e: lane r addresses
  // chunk r % 4 of token s0 + r / 4 and the transposing read deals the columns out
  template <typename F>
  static __device__ __forceinline__ Frag<bf16_t> col_frag(const char* t, int s0, int r, F col) {
    const int c = col(r & 3), row = s0 + (r >> 2);
    const uint2 lo = tiles::ld_tr(t + off(row, c >> 3) + ((c & 4) << 1));
    const uint2 hi = tiles::ld_tr(t + off(row + 4, c >> 3) + ((c & 4) << 1));
    Frag<bf16_t> f;
    f.v = __builtin_bit_cast(bf16x8, u32x4{lo.x, lo.y, hi.x, hi.y});
    return f;
  }
};
template <int COLS> struct Tile<float, COLS> {
  static constexpr int stride = COLS * 4 + 16;
  static constexpr int bytes = BT * stride;
  static constexpr int units = COLS / 4;
  static __device__ __forceinline__ int off(int row, int u) { return row * stride + 16 * u; }
  static __device__ __forceinline__ Frag<float> row_frag(const char* t, int row, int slab, int q) {
    Frag<float> f;
    load8(f, reinterpret_cast<const float*>(t + row * stride) + 32 * slab + 8 * q);
    return f;
  }
  template <typename F>
  static __device__ __forceinline__ Frag<float> col_frag(const char* t, int s0, int r, F col) {
    const int c = col(r >> 2) + (r & 3);
    Frag<float> f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = *reinterpret_cast<const float*>(t + (s0 + e) * stride + 4 * c);
    return f;
  }
};

// Two accumulators -> the operand slots 8 q + e (blocks numbered by perm_row).
__device__ __forceinline__ Frag<bf16_t> frag_of(f32x4 a, f32x4 b, bf16_t) {
  Frag<bf16_t> f;
  f.v = __builtin_bit_cast(bf16x8, u32x4{pack_bf2(a[0], a[1]), pack_bf2(a[2], a[3]), pack_bf2(b[0], b[1]),
                                         pack_bf2(b[2], b[3])});
  return f;
}
__device__ __forceinline__ Frag<float> frag_of(f32x4 a, f32x4 b, float) {
  Frag<float> f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f.v[i] = a[i];
    f.v[4 + i] = b[i];
  }
  return f;
}

__device__ __forceinline__ float ex2(float x) { return __builtin_amdgcn_exp2f(x); }

// ------------------------------------------------------------ gates
// Inclusive sum over the 64 lanes in fp64 by DPP (row shifts 1, 2, 4, 8, then
// the row totals of lanes 15 and 31 to the rows behind them).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_add(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return x + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double wave_scan(double x) {
  x = dpp_add<0x111, 0xF>(x);
  x = dpp_add<0x112, 0xF>(x);
  x = dpp_add<0x114, 0xF>(x);
  x = dpp_add<0x118, 0xF>(x);
  x = dpp_add<0x142, 0xA>(x);   // row_bcast:15 into rows 1 and 3
  x = dpp_add<0x143, 0xC>(x);   // row_bcast:31 into rows 2 and 3
  return x;
}
__device__ __forceinline__ double lane63(double x) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

struct Gates {              // of one chunk and head, in LDS
  float hi[BT], lo[BT];     // G_t as a pair
  float dt[BT];             // D_t
  float w[BT];              // D_t 2^{G_63 - G_t}
  float eg[BT];             // 2^{G_t}
};

// ------------------------------------------------------------ segments
struct Segment {
  int n, j;              // sequence (< 0: none), segment of it
  long long start;       // its sequence's first token among the batch row's
  int len;               // tokens of the sequence
};

// Which segment slot `slot` is.  Same result in every lane.
__device__ __forceinline__ Segment find_segment(const SsmArgs& a, int seg, int slot, int lane) {
  Segment g;
  if (!a.cu) {
    const int per = a.T > seg ? (a.T + seg - 1) / seg : 1;
    g.n = slot / per;
    g.j = slot - g.n * per;
    g.start = 0;
    g.len = a.T;
    return g;
  }
  g.n = -1;
  g.j = 0;
  g.start = 0;
  g.len = 0;
  int run = 0;
  for (int base = 0; base < a.N; base += 64) {
    const int n = base + lane;
    long long b0 = 0, b1 = 0;
    if (n < a.N) {
      b0 = a.cu[n];
      b1 = a.cu[n + 1];
      b0 = b0 < 0 ? 0 : (b0 > a.T ? a.T : b0);
      b1 = b1 < b0 ? b0 : (b1 > a.T ? a.T : b1);
    }
    const int len = (int)(b1 - b0);
    const int segs = n < a.N ? (len > seg ? (len + seg - 1) / seg : 1) : 0;
    int incl = segs;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(incl, off, 64);
      if (lane >= off) incl += y;
    }
    const int all = __builtin_amdgcn_readlane(incl, 63);
    if (slot < run + all) {
      const int l = __ffsll((unsigned long long)__ballot(incl > slot - run)) - 1;
      g.n = base + l;
      g.j = slot - run - (__builtin_amdgcn_readlane(incl, l) - __builtin_amdgcn_readlane(segs, l));
      g.start = __builtin_amdgcn_readlane((int)b0, l);
      g.len = __builtin_amdgcn_readlane(len, l);
      return g;
    }
    run += all;
  }
  return g;
}

// ------------------------------------------------------------ the scan
// OUT: the second (or only) launch, which writes y and ht; otherwise the first
// launch of a split call, which writes segment states and log-decays.
template <typename T, int K, int V, int NH, bool OUT>
__global__ __launch_bounds__(NT, sizeof(T) == 2 ? 2 : 1) void ssm_scan_kernel(
    SsmArgs a, int seg, int work, bool split, float* __restrict__ seg_state, double* __restrict__ seg_decay) {
  constexpr int CW = NH * V;            // columns of the work-group
  constexpr int NB = CW / 64;           // 16-column blocks of a wave
  constexpr int KB = K / 16, KS = K / 32;
  constexpr bool HALF = sizeof(T) == 2;
  typedef Tile<T, K> TK;
  typedef Tile<T, CW> TX;
  typedef Tile<T, BT> TM;
  __shared__ __align__(16) char sB[TK::bytes];
  __shared__ __align__(16) char sC[OUT ? TK::bytes : 16];
  __shared__ __align__(16) char sX[TX::bytes];
  __shared__ __align__(16) char sM[OUT ? NH * TM::bytes : 16];
  __shared__ Gates sG[2][NH];
  __shared__ float sDec[2][NH];

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  // heads of one segment (which share B and C) run next to each other on one XCD
  const int ht_count = a.HV / NH;
  const int per_xcd = (work + 7) / 8;
  const int id = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per_xcd || id >= work) return;
  const int slot = id / ht_count;
  const int hv0 = (id - slot * ht_count) * NH;
  const int hk = hv0 / (a.HV / a.Hk);
  const Segment sg = find_segment(a, seg, slot, lane);
  if (sg.n < 0) return;
  const int first = split ? sg.j * seg : 0;   // first token of the segment in its sequence
  const int stop = split && first + seg < sg.len ? first + seg : sg.len;
  const bool last = stop == sg.len;
  if (!OUT && last) return;                  // its state is nobody's start

  // rows of this sequence
  const long long brow = a.cu ? 0 : sg.n;
  const T* xp = reinterpret_cast<const T*>(a.x.p) + brow * a.x.batch + sg.start * a.x.token + (long long)hv0 * V;
  const T* bp = reinterpret_cast<const T*>(a.B.p) + brow * a.B.batch + sg.start * a.B.token + (long long)hk * K;
  const T* cp = reinterpret_cast<const T*>(a.C.p) + brow * a.C.batch + sg.start * a.C.token + (long long)hk * K;
  const T* dp = reinterpret_cast<const T*>(a.dt.p) + brow * a.dt.batch + sg.start * a.dt.token + hv0;

  // the lane's columns: block b holds column pcol(b) of the work-group's
  const int hw = NH == 2 ? w >> 1 : 0;       // the wave's head
  const int hv = hv0 + hw;
  auto pcol = [&](int b) { return NB == 2 ? 32 * w + 8 * (r >> 2) + 4 * b + (r & 3) : 16 * w + r; };
  auto pchunk = [&](int b, int c) { return NB == 2 ? 32 * w + 8 * c + 4 * b : 16 * w + 4 * c; };

  // ---- the starting state
  f32x4 S[KB][NB];
#pragma unroll
  for (int k = 0; k < KB; ++k)
#pragma unroll
    for (int b = 0; b < NB; ++b) S[k][b] = zero4();
  auto state_at = [&](long long entry, int b) -> size_t {   // element of the lane's (column, first channel)
    return (((size_t)entry * a.HV + hv) * V + (pcol(b) - hw * V)) * K + 8 * q;
  };
  auto add_state = [&](const float* base, long long entry, float f) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float* p = base + state_at(entry, b);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const f32x4 lo = *reinterpret_cast<const f32x4*>(p + 32 * k);
        const f32x4 hi = *reinterpret_cast<const f32x4*>(p + 32 * k + 4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          S[2 * k][b][i] = fmaf(f, lo[i], S[2 * k][b][i]);
          S[2 * k + 1][b][i] = fmaf(f, hi[i], S[2 * k + 1][b][i]);
        }
      }
    }
  };
  if (OUT) {
    // the segments before this one, nearest first; behind a decay that has
    // underflowed nothing is left to add
    double past = 0.0;
    float f = 1.0f;
    for (int i = 1; i <= sg.j && f != 0.0f; ++i) {
      add_state(seg_state, slot - i, f);
      past += seg_decay[(size_t)(slot - i) * a.HV + hv];
      f = ex2((float)past);
    }
    if (a.h0 && f != 0.0f) add_state(a.h0, sg.n, f);
  }

  // ---- staging: the next chunk's tiles in registers
  constexpr int UB = TK::units * BT / NT, UX = TX::units * BT / NT;
  u32x4 gB[UB], gC[OUT ? UB : 1], gX[UX];
  float gdt = 0.f;
  auto load_tiles = [&](int t0) {
    const int nr = stop - t0;
    const u32x4 none = {0, 0, 0, 0};
    if (w < NH) gdt = lane < nr ? to_f(dp[(long long)(t0 + lane) * a.dt.token + w]) : 0.f;
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      const int row = (tid + NT * i) / TK::units, u = (tid + NT * i) % TK::units;
      const bool in = row < nr;
      gB[i] = none;
      if (in) gB[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(bp + (t0 + row) * a.B.token) + 16 * u);
      if constexpr (OUT) {
        gC[i] = none;
        if (in) gC[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(cp + (t0 + row) * a.C.token) + 16 * u);
      }
    }
#pragma unroll
    for (int i = 0; i < UX; ++i) {
      const int row = (tid + NT * i) / TX::units, u = (tid + NT * i) % TX::units;
      gX[i] = none;
      if (row < nr)
        gX[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(xp + (t0 + row) * a.x.token) + 16 * u);
    }
  };
  auto put_tiles = [&]() {
#pragma unroll
    for (int i = 0; i < UB; ++i) {
      const int row = (tid + NT * i) / TK::units, u = (tid + NT * i) % TK::units;
      *reinterpret_cast<u32x4*>(sB + TK::off(row, u)) = gB[i];
      if constexpr (OUT) *reinterpret_cast<u32x4*>(sC + TK::off(row, u)) = gC[i];
    }
#pragma unroll
    for (int i = 0; i < UX; ++i) {
      const int row = (tid + NT * i) / TX::units, u = (tid + NT * i) % TX::units;
      *reinterpret_cast<u32x4*>(sX + TX::off(row, u)) = gX[i];
    }
  };

  // ---- gates of a chunk: wave h takes head h, a token per lane
  double A2 = 0.0, bias = 0.0, sum_decay = 0.0;
  if (w < NH) {
    A2 = -(double)expf(a.A_log[hv0 + w]) * 1.4426950408889634;
    bias = a.dt_bias ? a.dt_bias[hv0 + w] : 0.f;
  }
  auto gates = [&](int t0, int buf) {
    float d = gdt + (float)bias;
    if (a.softplus) d = d <= 20.f ? log1pf(expf(d)) : d;
    if (t0 + lane >= stop) d = 0.f;
    const double G = wave_scan((double)d * A2);
    const double tot = lane63(G);
    const float hi = (float)G;
    Gates& g = sG[buf][w];
    g.hi[lane] = hi;
    g.lo[lane] = (float)(G - (double)hi);
    g.dt[lane] = d;
    g.w[lane] = d * ex2((float)(tot - G));
    g.eg[lane] = ex2(hi);
    if (lane == 0) sDec[buf][w] = ex2((float)tot);
    sum_decay += tot;
  };

  const float skip = OUT && a.D ? a.D[hv] : 0.f;
  const bool fine = !OUT || (last && a.ht != nullptr);   // uniform: the state leaves the kernel

  load_tiles(first);
  if (w < NH) gates(first, 0);

  int buf = 0;
  for (int t0 = first; t0 < stop; t0 += BT, buf ^= 1) {
    const int nr = stop - t0 < BT ? stop - t0 : BT;
    tiles::lds_barrier();   // everyone has read the last chunk's tiles
    put_tiles();
    tiles::lds_barrier();
    const bool more = t0 + BT < stop;
    if (more) load_tiles(t0 + BT);
    const Gates& g = sG[buf][hw];

    // z of the lane's rows and columns (consecutive columns: 8, or 4)
    constexpr int CL = 4 * NB;
    const int p0 = NB == 2 ? 32 * w + 8 * q : 16 * w + 4 * q;
    float Yz[OUT ? 4 : 1][CL];
    u32x4 zr[OUT ? 4 : 1][CL * sizeof(T) > 16 ? 2 : 1];
    f32x4 Y[OUT ? 4 : 1][NB];
    if constexpr (OUT) {
      if (a.z.p) {
        const T* zp = reinterpret_cast<const T*>(a.z.p) + brow * a.z.batch + (sg.start + t0) * a.z.token +
                      (long long)hv0 * V + p0;
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const int t = perm_row(tb, r);
          if (t < nr) {
            const char* zt = reinterpret_cast<const char*>(zp + t * a.z.token);
            if constexpr (CL * sizeof(T) == 8) {
              const uint2 v = *reinterpret_cast<const uint2*>(zt);
              zr[tb][0] = u32x4{v.x, v.y, 0, 0};
            } else {
              zr[tb][0] = *reinterpret_cast<const u32x4*>(zt);
              if constexpr (CL * sizeof(T) == 32) zr[tb][1] = *reinterpret_cast<const u32x4*>(zt + 16);
            }
          }
        }
      }

      // ---- M of token block w: scores with tokens as columns, so that a lane
      // gets 8 consecutive s of one t
      {
        const int t = perm_row(w, r);
        Frag<T> ct[KS];
#pragma unroll
        for (int k = 0; k < KS; ++k) ct[k] = TK::row_frag(sC, t, k, q);
        for (int j = 0; j <= (w >> 1); ++j) {
          f32x4 e0 = zero4(), e1 = zero4();
#pragma unroll
          for (int k = 0; k < KS; ++k) {
            e0 = mma(TK::row_frag(sB, perm_row(2 * j, r), k, q), ct[k], e0);
            e1 = mma(TK::row_frag(sB, perm_row(2 * j + 1, r), k, q), ct[k], e1);
          }
          const int s0 = 32 * j + 8 * q;
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            const Gates& gh = sG[buf][h];
            const float th = gh.hi[t], tl = gh.lo[t];
            f32x4 m0, m1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int sa = s0 + i, sb = s0 + 4 + i;
              m0[i] = sa <= t ? e0[i] * gh.dt[sa] * ex2((th - gh.hi[sa]) + (tl - gh.lo[sa])) : 0.f;
              m1[i] = sb <= t ? e1[i] * gh.dt[sb] * ex2((th - gh.hi[sb]) + (tl - gh.lo[sb])) : 0.f;
            }
            char* row = sM + h * TM::bytes;
            const Frag<T> mf = frag_of(m0, m1, T());
            if constexpr (HALF) {
              *reinterpret_cast<bf16x8*>(row + TM::off(t, 4 * j + q)) = mf.v;
            } else {
              float* mp = reinterpret_cast<float*>(row + t * TM::stride) + s0;
              *reinterpret_cast<f32x4*>(mp) = m0;
              *reinterpret_cast<f32x4*>(mp + 4) = m1;
            }
          }
        }
      }

      // ---- Y^T = 2^{G_t} S C^T
#pragma unroll
      for (int tb = 0; tb < 4; ++tb)
#pragma unroll
        for (int b = 0; b < NB; ++b) Y[tb][b] = zero4();
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        Frag<T> sf[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) sf[b] = frag_of(S[2 * k][b], S[2 * k + 1][b], T());
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const Frag<T> cf = TK::row_frag(sC, perm_row(tb, r), k, q);
#pragma unroll
          for (int b = 0; b < NB; ++b) Y[tb][b] = mma(sf[b], cf, Y[tb][b]);
        }
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const float eg = g.eg[perm_row(tb, r)];
#pragma unroll
        for (int b = 0; b < NB; ++b) Y[tb][b] *= eg;
      }
    }

    // the next chunk's gates, in the waves that had the fewest scores
    if (more && w < NH) gates(t0 + BT, buf ^ 1);
    if constexpr (OUT) tiles::lds_barrier();   // M is complete

    // ---- x of the wave's columns; Y^T += x^T M^T
    const float dec = sDec[buf][hw];
#pragma unroll
    for (int k = 0; k < KB; ++k)
#pragma unroll
      for (int b = 0; b < NB; ++b) S[k][b] *= dec;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      Frag<T> xf[NB], x1[NB], x2[NB], x3[NB];
#pragma unroll
      for (int b = 0; b < NB; ++b) xf[b] = TX::col_frag(sX, 32 * j + 8 * q, r, [&](int c) { return pchunk(b, c); });
      if constexpr (OUT) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          if (j <= (tb >> 1)) {
            const Frag<T> mf = TM::row_frag(sM + hw * TM::bytes, perm_row(tb, r), j, q);
#pragma unroll
            for (int b = 0; b < NB; ++b) Y[tb][b] = mma(xf[b], mf, Y[tb][b]);
          }
        }
      }
      // ---- S += B^T (w o x)
      float ws[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) ws[e] = g.w[32 * j + 8 * q + e];
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        f32x4 lo, hi;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          lo[i] = xf[b].get(i) * ws[i];
          hi[i] = xf[b].get(4 + i) * ws[4 + i];
        }
        x1[b] = frag_of(lo, hi, T());
        if constexpr (HALF) {
          if (fine) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              lo[i] -= x1[b].get(i);
              hi[i] -= x1[b].get(4 + i);
            }
            x2[b] = frag_of(lo, hi, T());
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              lo[i] -= x2[b].get(i);
              hi[i] -= x2[b].get(4 + i);
            }
            x3[b] = frag_of(lo, hi, T());
          }
        }
      }
#pragma unroll
      for (int k = 0; k < KB; ++k) {
        const Frag<T> bf = TK::col_frag(sB, 32 * j + 8 * q, r,
                                        [&](int c) { return 32 * (k >> 1) + 4 * (k & 1) + 8 * c; });
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          S[k][b] = mma(bf, x1[b], S[k][b]);
          if constexpr (HALF) {
            if (fine) {
              S[k][b] = mma(bf, x2[b], S[k][b]);
              S[k][b] = mma(bf, x3[b], S[k][b]);
            }
          }
        }
      }
    }

    // ---- y
    if constexpr (OUT) {
      T* yp = reinterpret_cast<T*>(a.y) + ((brow * a.T + sg.start + t0) * a.HV + hv0) * (long long)V + p0;
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const int t = perm_row(tb, r);
#pragma unroll
        for (int e = 0; e < CL; ++e) Yz[tb][e] = Y[tb][e >> 2][e & 3];
        if (a.D) {
          float xv[CL];
          if constexpr (HALF) {
            const bf16_t* xr = reinterpret_cast<const bf16_t*>(sX + TX::off(t, p0 >> 3)) + (p0 & 7);
#pragma unroll
            for (int e = 0; e < CL; ++e) xv[e] = bf2f(xr[e]);
          } else {
            const float* xr = reinterpret_cast<const float*>(sX + TX::off(t, p0 >> 2));
#pragma unroll
            for (int e = 0; e < CL; ++e) xv[e] = xr[e];
          }
#pragma unroll
          for (int e = 0; e < CL; ++e) Yz[tb][e] = fmaf(skip, xv[e], Yz[tb][e]);
        }
        if (a.z.p) {
#pragma unroll
          for (int e = 0; e < CL; ++e) {
            float z;
            if constexpr (HALF) {
              const uint32_t wd = zr[tb][0][e >> 1];
              z = __builtin_bit_cast(float, (e & 1) ? wd & 0xFFFF0000u : wd << 16);
            } else {
              z = __builtin_bit_cast(float, (uint32_t)zr[tb][e >> 2][e & 3]);
            }
            Yz[tb][e] *= z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
          }
        }
        if (t < nr) {
          T* yt = yp + (long long)t * a.HV * V;
          if constexpr (HALF && NB == 2) {
            *reinterpret_cast<u32x4*>(yt) =
                u32x4{pack_bf2(Yz[tb][0], Yz[tb][1]), pack_bf2(Yz[tb][2], Yz[tb][3]), pack_bf2(Yz[tb][4], Yz[tb][5]),
                      pack_bf2(Yz[tb][6], Yz[tb][7])};
          } else if constexpr (HALF) {
            *reinterpret_cast<uint2*>(yt) = uint2{pack_bf2(Yz[tb][0], Yz[tb][1]), pack_bf2(Yz[tb][2], Yz[tb][3])};
          } else {
#pragma unroll
            for (int e = 0; e < CL; e += 4)
              *reinterpret_cast<f32x4*>(yt + e) = f32x4{Yz[tb][e], Yz[tb][e + 1], Yz[tb][e + 2], Yz[tb][e + 3]};
          }
        }
      }
    }
  }

  // ---- the final state
  float* dst = OUT ? a.ht : seg_state;
  if (OUT ? (last && a.ht != nullptr) : true) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float* p = dst + state_at(OUT ? sg.n : slot, b);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        *reinterpret_cast<f32x4*>(p + 32 * k) = S[2 * k][b];
        *reinterpret_cast<f32x4*>(p + 32 * k + 4) = S[2 * k + 1][b];
      }
    }
  }
  if (!OUT && w < NH && lane == 0) seg_decay[(size_t)slot * a.HV + hv0 + w] = sum_decay;
}

template <typename T, int K, int V, int NH>
hipError_t launch_t(const SsmArgs& a, const SsmPlan& p, hipStream_t s) {
  const int work = p.slots * (a.HV / NH);
  const dim3 grid((unsigned)((work + 7) / 8 * 8)), block(NT);
  float* st = reinterpret_cast<float*>(a.workspace);
  double* dec = p.split ? reinterpret_cast<double*>(reinterpret_cast<char*>(a.workspace) + p.decay_off) : nullptr;
  if (p.split) {
    hipLaunchKernelGGL((ssm_scan_kernel<T, K, V, NH, false>), grid, block, 0, s, a, p.seg, work, true, st, dec);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((ssm_scan_kernel<T, K, V, NH, true>), grid, block, 0, s, a, p.seg, work, p.split, st, dec);
  return hipGetLastError();
}

template <typename T>
hipError_t launch_io(const SsmArgs& a, const SsmPlan& p, hipStream_t s) {
  if (a.V == 128) return a.K == 128 ? launch_t<T, 128, 128, 1>(a, p, s) : launch_t<T, 64, 128, 1>(a, p, s);
  if (p.nh == 2) return a.K == 128 ? launch_t<T, 128, 64, 2>(a, p, s) : launch_t<T, 64, 64, 2>(a, p, s);
  return a.K == 128 ? launch_t<T, 128, 64, 1>(a, p, s) : launch_t<T, 64, 64, 1>(a, p, s);
}

}  // namespace

SsmPlan ssm_plan(int nb, int T, int Hk, int HV, int K, int V, int N, bool varlen, bool bf16) {
  SsmPlan p;
  // two 64-wide heads of one group share their scores
  p.nh = V == 64 && (HV / Hk) % 2 == 0 ? 2 : 1;
  const long long tokens = (long long)nb * T;
  const long long tiles = HV / p.nh;
  // work-groups resident on 256 CUs: two a CU, one with fp32 tiles
  const long long want = bf16 ? 512 : 256;
  long long seg = ((tokens * tiles + want - 1) / want + 63) / 64 * 64;
  seg = seg < 256 ? 256 : seg;
  if (seg >= T) seg = ((long long)T + 63) / 64 * 64;
  p.split = seg < T;
  p.seg = seg > 64 ? (int)seg : 64;
  p.slots = !p.split ? N : (varlen ? (int)(tokens / seg) + N : N * (int)((T + seg - 1) / seg));
  const size_t state = (size_t)p.slots * HV * V * K * 4;
  p.decay_off = (state + 255) / 256 * 256;
  p.bytes = p.split ? p.decay_off + ((size_t)p.slots * HV * 8 + 255) / 256 * 256 : 0;
  return p;
}

hipError_t launch_ssm_fwd(const SsmArgs& a, hipStream_t s) {
  const SsmPlan p = ssm_plan(a.nb, a.T, a.Hk, a.HV, a.K, a.V, a.N, a.cu != nullptr, a.bf16 != 0);
  return a.bf16 ? launch_io<bf16_t>(a, p, s) : launch_io<float>(a, p, s);
}

}  // namespace gdn
