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
// Work is cut into (sequence segment, 64 or 128 value columns).  A work-group walks
// the chunks of its segment with the state in accumulators: each of its 4 waves owns
// 16 or 32 columns and all K channels, so S^T feeds both products from registers.
// The scores C B^T, 12 blocks of 16 x 16 on and under the diagonal, are dealt out
// three to a wave (with tokens as columns they leave the matrix core as the operand
// of the next product), gated for each head and passed through LDS.  Gates come in
// groups: each wave computes those of one chunk and head, a token per lane, for the
// next 2 or 4 chunks at once (a chain of exponentials and 64-bit sums that one or
// two waves would have everyone else wait for at every chunk).  Tiles arrive by
// direct-to-LDS loads into one buffer: up to 69 KiB a work-group in bf16 at K = 128,
// two work-groups a CU (two waves a SIMD), which hide each other's latencies.  Eight
// waves of 16 columns took the same time: more waves to hide latency, but every
// fragment of B, C and M read from LDS twice as often.  Where sequences x heads are
// too few for the chip, sequences are split: a first launch computes each segment's
// own final state (from zeros) and log-decay, a second one joins them with h0 in
// order, and the third starts each segment from the state behind the one before.
// That reads x and B twice but moves no per-chunk states.
//
// Measured (bf16, K = 128; a call's time from captured calls over three inputs in turn,
// the launches' from a kernel trace of warm calls, which adds up to 4 %).  One prompt
// of 8192 tokens x 64 heads of 64, gated: launches of 38 + 13 + 70 us, 118 a call for
// 209 MB (41 us at a large copy's 5.1 TB/s).  Eight packed prompts of 5003 tokens, 32
// heads of 128, initial and final states: 31 + 12 + 49 us, 92 a call, 136 MB (27 us).
// The same 8192 tokens as 16 prompts, one launch: 82 us a call.  fp32, 4096 tokens x 32
// heads of 64: 31 + 8 + 80 us, 114 a call, 106 MB (21 us; its products take about 56).
// What bounds it is no one unit: of the last launch's cycles the vector ALU issues in
// 41 %, LDS in 19 % with 11 % more of bank conflicts (the transposing reads and the
// stores of M take one half of every 16-byte unit at a time, so half of the banks), the
// matrix cores work in 13 %, between three barriers a chunk: with two waves a SIMD the
// latencies of the tiles and of z are only partly hidden.  Twice the waves gained
// nothing, nor did a higher wave priority for the products.  The first launch takes 13
// us without its state update, 29 with one bf16 term of three.
//
// Precision.  Gate sums are taken in 64 bits, over log2-decays held at -160 a
// token or more (2^-160 is 0 in fp32 already), so that with bf16 io an fp32 G is
// good to 10240 x 2^-24 = 2^-10.7 at worst; with fp32 io G is an fp32 pair, whose
// differences keep their last places.  A state that leaves the kernel (ht, and a
// segment's state handed on) is formed from the exact products of B with the
// scaled x as three bf16 terms (24 bits); the state that only feeds this
// segment's bf16 y takes one term, and S and M are rounded to bf16 as operands.
// (x, B and C may be of any size, so fp16 with its 11 bits does not do; a second term
// of S and M would cost half again of the products and 16 KiB more for M, with which
// two work-groups no longer fit a CU.)  y of the workloads above is off by 0.0018 and
// 0.0019 of its norm against 64 bits, of which storing y as bf16 makes 0.0017.

#include <math.h>

#include "gdn_device.h"
#include "mixer_launch.h"
#include "scan_tiles.h"
#include "ssm_rate.h"

namespace gdn {

namespace {

using tiles::BT;
using tiles::perm_row;
using tiles::u32x4;

constexpr int NW = 4;   // waves of a work-group

// ------------------------------------------------------------ LDS tiles
// A tile of 64 rows (tokens) by COLS in 16-byte units swizzled by row: for bf16 as
// in scan_tiles.h (row fragments and transposing reads are conflict-free).  The
// swizzle of a row is the same 4 and 32 rows further, and it is an XOR of the unit,
// so one address a lane serves a whole tile: token blocks and halves are immediate
// offsets, the 32-channel slab `k` an XOR with k * slab_x.
template <typename T, int COLS> struct Tile;
template <int COLS> struct Tile<bf16_t, COLS> {
  static constexpr int row_bytes = COLS * 2, bytes = BT * row_bytes, slab_x = 64;
  static constexpr int units = COLS / 8;   // 16-byte units of a row
  static __device__ __forceinline__ int off(int row, int u) { return tiles::qk_off<COLS>(row, u); }
  // slots 8 q + e of row perm_row(0, r)
  static __device__ __forceinline__ int row_at(int r, int q) { return off(perm_row(0, r), q); }
  // ... of row perm_row(blk, r)
  static __device__ __forceinline__ Frag<bf16_t> row_frag(const char* t, int at, int blk) {
    Frag<bf16_t> f;
    f.v = *reinterpret_cast<const bf16x8*>(t + at + tiles::blk_rows(blk) * row_bytes);
    return f;
  }
  // Tokens 8 q + e of column col(r / 4) + r % 4: lane r addresses the 4-column
  // chunk r % 4 of token r / 4 and the transposing read deals the columns out.
  struct Col { int at; };
  template <typename F>
  static __device__ __forceinline__ Col col_at(int r, int q, F col) {
    const int c = col(r & 3);
    return Col{off(8 * q + (r >> 2), c >> 3) + ((c & 4) << 1)};
  }
  // ... of tokens 32 j + 8 q + e, of the columns 4 further (half = 1) in slab k
  static __device__ __forceinline__ Frag<bf16_t> col_frag(const char* t, const Col& c, int j, int k, int half) {
    const char* p = t + (c.at ^ (k * slab_x)) + 32 * j * row_bytes + 8 * half;
    const uint2 lo = tiles::ld_tr(p);
    const uint2 hi = tiles::ld_tr(p + 4 * row_bytes);
    Frag<bf16_t> f;
    f.v = __builtin_bit_cast(bf16x8, u32x4{lo.x, lo.y, hi.x, hi.y});
    return f;
  }
  // ... of the 16 columns 16 n further, where col(i) = 4 i
  static __device__ __forceinline__ Frag<bf16_t> col_blk(const char* t, const Col& c, int j, int n) {
    return col_frag(t, Col{c.at ^ (n * (slab_x / 2))}, j, 0, 0);
  }
};
template <int COLS> struct Tile<float, COLS> {
  static constexpr int row_bytes = COLS * 4, bytes = BT * row_bytes, slab_x = 128;
  static constexpr int units = COLS / 4;
  static __device__ __forceinline__ int swz(int row) { return (((row & 3) << 1) | (((row >> 3) & 3) << 3)) & (units - 1); }
  static __device__ __forceinline__ int off(int row, int u) { return row * row_bytes + ((u ^ swz(row)) << 4); }
  static __device__ __forceinline__ int row_at(int r, int q) { return off(perm_row(0, r), 2 * q); }
  static __device__ __forceinline__ Frag<float> row_frag(const char* t, int at, int blk) {
    const char* p = t + at + tiles::blk_rows(blk) * row_bytes;   // the swizzle leaves a unit's lowest bit alone
    const f32x4 a = *reinterpret_cast<const f32x4*>(p);
    const f32x4 b = *reinterpret_cast<const f32x4*>(p + 16);
    Frag<float> f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.v[i] = a[i];
      f.v[4 + i] = b[i];
    }
    return f;
  }
  struct Col { int at[4]; };
  template <typename F>
  static __device__ __forceinline__ Col col_at(int r, int q, F col) {
    const int c = col(r >> 2) + (r & 3);
    Col k;
#pragma unroll
    for (int e = 0; e < 4; ++e) k.at[e] = off(8 * q + e, c >> 2) + 4 * (c & 3);
    return k;
  }
  static __device__ __forceinline__ Frag<float> col_frag(const char* t, const Col& c, int j, int k, int half) {
    Frag<float> f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f.v[e] = *reinterpret_cast<const float*>(t + (c.at[e & 3] ^ (k * slab_x)) + (32 * j + 4 * (e >> 2)) * row_bytes + 16 * half);
    return f;
  }
  static __device__ __forceinline__ Frag<float> col_blk(const char* t, const Col& c, int j, int n) {
    Frag<float> f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f.v[e] = *reinterpret_cast<const float*>(t + (c.at[e & 3] ^ (n * (slab_x / 2))) + (32 * j + 4 * (e >> 2)) * row_bytes);
    return f;
  }
};

// Direct-to-LDS copy of a tile: a wave's load i brings 1 KiB, RPL whole rows from
// row NW RPL i + w RPL on.  Rows past the sequence's end repeat its last row (their
// weights are 0).  The lane offsets are computed anew for every chunk (the asm sees
// to it): a few instructions against six registers held over the loop.
template <typename T, int COLS>
__device__ __forceinline__ void load_tile(const char* src, uint32_t stride, char* tile, int nr, int w, int lane) {
  typedef Tile<T, COLS> TL;
  constexpr int RPL = 64 / TL::units, N = BT / RPL / NW, H = N >= 2 ? N / 2 : 1;   // H: loads of 32 rows
  tiles::lchar* dst = (tiles::lchar*)tile + w * 1024;
  int l = lane;
  asm volatile("" : "+v"(l));
  const int t0 = w * RPL + l / TL::units;
  if (nr >= BT) {   // the swizzle repeats every 32 rows, and so do the lane offsets
    uint32_t off[H];
#pragma unroll
    for (int i = 0; i < H; ++i) {
      const int t = t0 + NW * RPL * i;
      off[i] = (uint32_t)t * stride + (uint32_t)(TL::off(t, l % TL::units) - t * TL::row_bytes);
    }
#pragma unroll
    for (int h = 0; h < N / H; ++h) {
      const char* sh = src + (uint64_t)stride * (uint32_t)(32 * h);
      asm volatile("" : "+s"(sh));
#pragma unroll
      for (int i = 0; i < H; ++i) tiles::dma16(sh + off[i], dst + (h * H + i) * (NW * 1024));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = t0 + NW * RPL * i;
      const uint32_t u = (uint32_t)(TL::off(t, l % TL::units) - t * TL::row_bytes);
      tiles::dma16(src + ((uint32_t)(t < nr ? t : nr - 1) * stride + u), dst + i * (NW * 1024));
    }
  }
}

// Global memory by pointers whose origin the compiler cannot see (below): as flat
// accesses they would count among the LDS ones, and every wait for an LDS read would
// wait for them.
template <typename V>
__device__ __forceinline__ V gload(const char* p) {
  typedef V U __attribute__((aligned(sizeof(V) < 16 ? sizeof(V) : 16)));
  return *(const __attribute__((address_space(1))) U*)p;
}
template <typename V>
__device__ __forceinline__ void gstore(char* p, V v) {
  typedef V U __attribute__((aligned(sizeof(V) < 16 ? sizeof(V) : 16)));
  *(__attribute__((address_space(1))) U*)p = v;
}

// The same through registers.
template <typename T, int COLS>
struct StageTile {
  typedef Tile<T, COLS> TL;
  static constexpr int RPL = 64 / TL::units, N = BT / RPL / NW;
  u32x4 v[N];
  __device__ __forceinline__ void load(const char* src, uint32_t stride, int w, int lane, int nr) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      int t = (NW * i + w) * RPL + lane / TL::units;
      if (nr < BT) t = t < nr ? t : nr - 1;   // rows past the end repeat the last one
      v[i] = gload<u32x4>(src + ((uint32_t)t * stride + 16u * (uint32_t)(lane % TL::units)));
    }
  }
  __device__ __forceinline__ void put(char* tile, int w, int lane) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int t = (NW * i + w) * RPL + lane / TL::units;
      *reinterpret_cast<u32x4*>(tile + TL::off(t, lane % TL::units)) = v[i];
    }
  }
};

// A uniform pointer that walks down the rows of an operand, 64 at a time.  The
// empty asm keeps the compiler from folding it into per-lane 64-bit addresses:
// base in scalar registers, 32-bit lane offsets.
struct Walk {
  const char* p;
  uint32_t stride;   // bytes of a row
  __device__ __forceinline__ void init(const Rows& r, long long brow, long long row, long long first, int elem) {
    p = reinterpret_cast<const char*>(r.p) + (brow * r.batch + row * r.token + first) * elem;
    stride = (uint32_t)r.token * (uint32_t)elem;
  }
  __device__ __forceinline__ const char* at(int row) const {   // uniform row
    const char* x = p + (uint64_t)stride * (uint32_t)row;
    asm volatile("" : "+s"(x));
    return x;
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

// Waits until at most N memory accesses of the wave are in flight.
template <int N>
__device__ __forceinline__ void wait_vm() {
  __builtin_amdgcn_s_waitcnt((N & 15) | (N >> 4) << 14 | 0x0F70);
}

// Fragments are read from LDS one product ahead of their use: left alone, the compiler
// has every product wait for its own (200 packed prompts of 60 tokens x 64 heads 282 ->
// 278 us, 100 tokens x 8 heads 16.3 -> 16.0, the long prompt above the same, the packed
// ones 91 -> 92).  LDS accesses stay on their side of this, everything else may cross.
__device__ __forceinline__ void ahead() { __builtin_amdgcn_sched_barrier(1); }

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
__device__ __forceinline__ double lane_of(double x, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, x);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, l);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), l);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

constexpr double LOG2E = 1.4426950408889634;

// Gates of a chunk and head, in LDS.  Scores are gated by 2^{G_t - G_s} D_s.
template <bool HALF> struct alignas(16) Gates {
  float g[BT];            // G_t
  float e[BT];            // G_s - log2 D_s (bf16 io); D_s (fp32 io)
  float w[BT];            // D_t 2^{G_63 - G_t}
  float eg[BT];           // 2^{G_t}
  float lo[HALF ? 4 : BT];   // what g leaves of G_t (fp32 io)
};

// ------------------------------------------------------------ y, z and x rows
// The lane's four or eight consecutive columns of a row.
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
template <int BYTES> struct VecOf;
template <> struct VecOf<8> { typedef u32x2 type; };
template <> struct VecOf<16> { typedef u32x4 type; };
template <> struct VecOf<32> { typedef u32x8 type; };

template <typename T, typename V>
__device__ __forceinline__ float elem(const V& v, int e) {
  if constexpr (sizeof(T) == 2) {
    const uint32_t w = v[e >> 1];
    return __builtin_bit_cast(float, (e & 1) ? w & 0xFFFF0000u : w << 16);
  } else {
    return __builtin_bit_cast(float, (uint32_t)v[e]);
  }
}
// from a tile: one 16-byte unit (or half of one), or two neighbours
template <typename V>
__device__ __forceinline__ V lds_vec(const char* p) {
  if constexpr (sizeof(V) == 32) {
    const u32x4 a = *reinterpret_cast<const u32x4*>(p), b = *reinterpret_cast<const u32x4*>(p + 16);
    return V{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
  } else {
    return *reinterpret_cast<const V*>(p);
  }
}
template <int N>
__device__ __forceinline__ typename VecOf<2 * N>::type pack(const float (&y)[N], bf16_t) {
  if constexpr (N == 8) return u32x4{pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3]), pack_bf2(y[4], y[5]), pack_bf2(y[6], y[7])};
  else return u32x2{pack_bf2(y[0], y[1]), pack_bf2(y[2], y[3])};
}
template <int N>
__device__ __forceinline__ typename VecOf<4 * N>::type pack(const float (&y)[N], float) {
  typename VecOf<4 * N>::type v;
#pragma unroll
  for (int e = 0; e < N; ++e) v[e] = __builtin_bit_cast(uint32_t, y[e]);
  return v;
}

// ------------------------------------------------------------ segments
struct Segment {
  int n, j;              // sequence (< 0: none), segment of it
  int state;             // its state in the workspace, if the sequence is split
  long long start;       // its sequence's first token among the batch row's
  int len;               // tokens of the sequence
};

// Tokens [b0, b0 + len) of packed sequence n.
struct Bounds {
  long long b0;
  int len;
  __device__ __forceinline__ Bounds(const SsmArgs& a, int n) {
    b0 = a.cu[n];
    long long b1 = a.cu[n + 1];
    b0 = b0 < 0 ? 0 : (b0 > a.T ? a.T : b0);
    b1 = b1 < b0 ? b0 : (b1 > a.T ? a.T : b1);
    len = (int)(b1 - b0);
  }
};

// States of packed sequence n in the workspace: one a segment, none for a single one.
__device__ __forceinline__ int states_of(const SsmArgs& a, int seg, int n) {
  if (n >= a.N) return 0;
  const int len = Bounds(a, n).len;
  return len > seg ? (len + seg - 1) / seg : 0;
}

// Inclusive sum over the lanes, and that of all.
struct LaneSum {
  int incl, all;
  __device__ __forceinline__ LaneSum(int x, int lane) {
    incl = x;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int y = __shfl_up(incl, off, 64);
      if (lane >= off) incl += y;
    }
    all = __builtin_amdgcn_readlane(incl, 63);
  }
};

// A packed sequence that is split, written by the join for the last launch: its
// number, its first state and its states (0: there is no such sequence).
struct alignas(16) SplitSeq {
  int n, state, states, unused;
};

// The segment and head tile of work-group `wg` of 8 XCDs: the tiles of a segment
// (which share B and C) run next to each other on one XCD, and every XCD gets an
// equal run of the segments that there are (packed sequences seldom fill the slots
// the host counts).  Same result in every lane; n < 0: none.
// First launch (few work-groups): the segments with a state, by the boundaries of all
// sequences, 64 at a time.  Last launch (one work-group for every sequence and tile at
// least): all segments, by the table of the split sequences, which are few; looking
// through all boundaries here too took 4.2 ms for 4096 prompts of 64 tokens x 16
// heads, this 0.64 ms.
template <bool OUT>
__device__ __forceinline__ Segment find_segment(const SsmArgs& a, int seg, int slots, bool split,
                                                const SplitSeq* table, int joins, int tiles, int wg, int lane,
                                                int& tile) {
  Segment g;
  g.n = -1;
  g.j = g.state = 0;
  g.start = 0;
  g.len = 0;
  int slot;
  auto deal = [&](int slots) -> bool {
    const int work = slots * tiles, per_xcd = (work + 7) / 8;
    const int id = (wg & 7) * per_xcd + (wg >> 3);
    slot = id / tiles;
    tile = id - slot * tiles;
    return (wg >> 3) < per_xcd && id < work;
  };
  if (!a.cu) {
    if (!deal(slots)) return g;
    const int per = a.T > seg ? (a.T + seg - 1) / seg : 1;
    g.n = slot / per;
    g.j = slot - g.n * per;
    g.state = slot;
    g.len = a.T;
    return g;
  }
  if constexpr (OUT) {
    int used = a.N;
    SplitSeq e{};
    auto read = [&](int base) {
      e.states = 0;
      if (base + lane < joins) e = table[base + lane];
    };
    if (split) {
      for (int base = 0; base < joins; base += 64) {
        read(base);
        used += LaneSum(e.states > 1 ? e.states - 1 : 0, lane).all;
      }
    }
    if (!deal(used < slots ? used : slots)) return g;   // boundaries out of order may claim more
    int n = slot;
    if (split) {
      for (int base = 0; base < joins; base += 64) {
        if (joins > 64) read(base);
        // segments of the sequences in front of a split one: one each, and the others
        // (states less sequences) of the split ones among them
        const int first = e.n + e.state - (base + lane);
        const unsigned long long before = __ballot(e.states > 0 && first <= slot);
        if (before == 0) break;
        const int l = 63 - __clzll((long long)before);
        const int at = slot - __builtin_amdgcn_readlane(first, l), of = __builtin_amdgcn_readlane(e.states, l);
        n = __builtin_amdgcn_readlane(e.n, l) + (at < of ? 0 : at - of + 1);
        g.j = at < of ? at : 0;
        g.state = __builtin_amdgcn_readlane(e.state, l) + g.j;
      }
    }
    if (n < 0 || n >= a.N) return g;
    g.n = n;
  } else {
    int st = states_of(a, seg, lane);
    LaneSum sum(st, lane);
    int used = sum.all;
    for (int base = 64; base < a.N; base += 64) used += LaneSum(states_of(a, seg, base + lane), lane).all;
    if (!deal(used < slots ? used : slots)) return g;
    int run = 0;   // of the sequences before these 64
    for (int base = 0; base < a.N; base += 64) {
      if (base > 0) {
        st = states_of(a, seg, base + lane);
        sum = LaneSum(st, lane);
      }
      if (slot < run + sum.all) {
        const int l = __ffsll((unsigned long long)__ballot(sum.incl > slot - run)) - 1;
        g.n = base + l;
        g.j = slot - run - __builtin_amdgcn_readlane(sum.incl - st, l);
        g.state = slot;
        break;
      }
      run += sum.all;
    }
    if (g.n < 0) return g;
  }
  const Bounds s(a, g.n);
  g.start = s.b0;
  g.len = s.len;
  return g;
}

// ------------------------------------------------------------ the scan
// OUT: the last (or only) launch, which writes y and ht; otherwise the first
// launch of a split call, which writes segment states and log-decays.
template <typename T, int K, int V, int NH, bool OUT>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 2 ? 2 : 1) void ssm_scan_kernel(
    SsmArgs a, int seg, int slots, int states, bool split, const SplitSeq* __restrict__ table, int joins,
    float* __restrict__ seg_state, double* __restrict__ seg_decay) {
  constexpr int CW = NH * V;            // columns of the work-group
  constexpr int NB = CW / 16 / NW;      // 16-column blocks of a wave
  constexpr int KB = K / 16, KS = K / 32;
  constexpr bool HALF = sizeof(T) == 2;   // bf16 io
  typedef Tile<T, K> TK;
  typedef Tile<T, CW> TX;
  typedef Tile<T, BT> TM;
  __shared__ __align__(16) char sB[TK::bytes];
  __shared__ __align__(16) char sC[OUT ? TK::bytes : 16];
  __shared__ __align__(16) char sX[TX::bytes];
  __shared__ __align__(16) char sM[OUT ? NH * TM::bytes : 16];
  constexpr int GC = NW / NH;           // chunks of a group of gates
  __shared__ Gates<HALF> sG[GC][NH];
  __shared__ float sDec[GC][NH];
  __shared__ double sSum[NW];           // log2-decay of the chunks whose gates the wave computed

  const int tid = threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r = lane & 15, q = lane >> 4;
  int tile;
  const Segment sg = find_segment<OUT>(a, seg, OUT ? slots : states, split, table, joins, a.HV / NH, blockIdx.x,
                                       lane, tile);
  if (sg.n < 0) return;
  const int hv0 = tile * NH;
  const int hk = hv0 / (a.HV / a.Hk);
  const int first = split ? sg.j * seg : 0;   // first token of the segment in its sequence
  const int stop = split && first + seg < sg.len ? first + seg : sg.len;
  const bool last = stop == sg.len;
  // a sequence of one segment needs no join; elsewhere the last segment's state is
  // nobody's start and made only for ht
  const bool alone = !split || sg.len <= seg;
  if (!OUT && last && !a.ht) return;

  // rows of this sequence, from the segment's first on
  const long long brow = a.cu ? 0 : sg.n;
  const long long row0 = sg.start + first;
  Walk wx, wb, wc, wz, wd, wy;
  wx.init(a.x, brow, row0, (long long)hv0 * V, sizeof(T));
  wb.init(a.B, brow, row0, (long long)hk * K, sizeof(T));
  wc.init(a.C, brow, row0, (long long)hk * K, sizeof(T));
  wz.init(a.z, brow, row0, (long long)hv0 * V, sizeof(T));
  wd.init(a.dt, brow, row0, hv0, sizeof(T));
  wy.init(Rows{a.y, (long long)a.T * a.HV * V, (long long)a.HV * V}, brow, row0, (long long)hv0 * V, sizeof(T));
  const int count = stop - first;   // tokens of the segment

  const int hw = 16 * NB * w / V;   // the wave's head
  const int hv = hv0 + hw;

  // ---- the starting state: lane (r, q) holds column col(b), channels
  // 32 k + 8 q + 0 .. 7 in S[2 k][b] and S[2 k + 1][b].  Two blocks of a wave are
  // interleaved so that the lanes' accumulator rows are 8 consecutive columns.  The
  // first launch, which makes no y, has its blocks of 16 columns and channels in order:
  // transposing reads then take whole units, without bank conflicts.
  auto col = [&](int b) { return OUT && NB == 2 ? 32 * w + 8 * (r >> 2) + 4 * b + (r & 3) : 16 * (NB * w + b) + r; };
  f32x4 S[KB][NB];
#pragma unroll
  for (int k = 0; k < KB; ++k)
#pragma unroll
    for (int b = 0; b < NB; ++b) S[k][b] = zero4();
  auto state_at = [&](long long entry, int b) -> size_t {
    return (((size_t)entry * a.HV + hv) * V + (col(b) - hw * V)) * K + (OUT ? 8 : 4) * q;
  };
  auto load_state = [&](const float* base, long long entry) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const float* p = base + state_at(entry, b);
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        S[2 * k][b] = *reinterpret_cast<const f32x4*>(p + 32 * k);
        S[2 * k + 1][b] = *reinterpret_cast<const f32x4*>(p + 32 * k + 4);
      }
    }
  };
  if (OUT) {
    if (sg.j > 0) {   // the joined state behind the segment before
      if (sg.state <= states) load_state(seg_state, sg.state - 1);   // always, for boundaries in order
    } else if (a.h0) {
      load_state(a.h0, sg.n);
    }
  }

  // ---- a chunk's tiles
  auto load_tiles = [&](int t0) {
    const int nr = count - t0;
    load_tile<T, K>(wb.at(t0), wb.stride, sB, nr, w, lane);
    load_tile<T, K>(wc.at(t0), wc.stride, sC, nr, w, lane);
    load_tile<T, CW>(wx.at(t0), wx.stride, sX, nr, w, lane);
  };
  // The first launch has the registers to hold the next chunk's tiles while it
  // computes.
  StageTile<T, K> gB;
  StageTile<T, CW> gX;
  auto stage = [&](int t0) {
    gB.load(wb.at(t0), wb.stride, w, lane, count - t0);
    gX.load(wx.at(t0), wx.stride, w, lane, count - t0);
  };

  // ---- gates of the wave's chunk and head of a group, a token per lane
  const int gc = w / NH, gh = w - gc * NH;
  T gdt{};   // raw dt, loaded a group ahead
  auto load_dt = [&](int t0) {   // t0: first token of the group
    const int t = t0 + BT * gc + lane;
    gdt = gload<T>(wd.at(0) + (uint64_t)(uint32_t)(t < count ? t : 0) * wd.stride + gh * (int)sizeof(T));
  };
  if (lane == 0) sSum[w] = 0.0;   // written and read by this wave only, up to the end
  const float A_log = a.A_log[hv0 + gh];
  const double A2 = -rate_of(A_log) * LOG2E;
  const bool fast = a.softplus && A_log > FAST_RATE;
  const float dt_bias = a.dt_bias ? a.dt_bias[hv0 + gh] : 0.f;
  auto gates = [&](int t0) {
    const float u = to_f(gdt) + dt_bias;
    float d = u;
    if (a.softplus) d = u <= 20.f ? log1pf(expf(u)) : u;
    double lg = (double)d * A2;
    if (fast) lg = -fast_decay(A_log, u) * LOG2E;
    lg = lg < -160.0 ? -160.0 : lg;
    if (t0 + BT * gc + lane >= count) {   // rows past the end leave the state alone
      d = 0.f;
      lg = 0.0;
    }
    const double G = wave_scan(lg);
    const double tot = lane_of(G, 63);
    Gates<HALF>& g = sG[gc][gh];
    const float hi = (float)G;
    if constexpr (OUT) {
      g.g[lane] = hi;
      if constexpr (HALF) {
        g.e[lane] = hi - __builtin_amdgcn_logf(d);   // +inf where D is 0
      } else {
        g.e[lane] = d;
        g.lo[lane] = (float)(G - (double)hi);
      }
      g.eg[lane] = ex2(hi);
    }
    g.w[lane] = d * ex2((float)(tot - G));
    if (lane == 0) {
      sDec[gc][gh] = ex2((float)tot);
      sSum[w] += tot;
    }
  };

  const float skip = OUT && a.D ? a.D[hv] : 0.f;
  // uniform: the state leaves the kernel (the join writes a split sequence's ht)
  const bool out_ht = OUT && alone && a.ht != nullptr;
  const bool fine = !OUT || out_ht;

  constexpr int CL = 4 * NB;        // consecutive columns of the lane in y, z and x
  typedef typename VecOf<CL * sizeof(T)>::type yvec;

  // The first launch walks its chunks backwards: with the decays of the chunks behind
  // in the weights, the state only grows and is not scaled 64 registers at a time.
  const int chunks = (count + BT - 1) / BT;
  const int c0 = OUT ? 0 : chunks - 1;
  float after = 1.f;   // decay of the chunks behind
  if (count > 0) {
    if constexpr (OUT) load_tiles(0);
    else stage(c0 * BT);
    load_dt(c0 / GC * GC * BT);
  }
  if constexpr (OUT) wait_vm<0>();

  for (int i = 0; OUT ? chunks > 0 : i < chunks; ++i) {
    const int t0 = (OUT ? i : c0 - i) * BT;
    const int buf = (t0 / BT) % GC;   // chunk of the group
    const int nr = count - t0 < BT ? count - t0 : BT;
    const bool more = i + 1 < chunks;
    const bool enter = OUT ? buf == 0 : i == 0 || buf == GC - 1;
    if (enter) gates(t0 - buf * BT);
    if constexpr (OUT) {
      // This wave's share of the tiles: behind its loads lie only the stores of the
      // chunk before, four or more.  With every wait where the compiler can count what
      // is behind it, it adds none for these stores, or for the next tiles below.
      wait_vm<4>();
    } else {
      gB.put(sB, w, lane);
      gX.put(sX, w, lane);
    }
    tiles::lds_barrier();
    if constexpr (OUT) {
      if (enter && t0 + GC * BT < count) load_dt(t0 + GC * BT);
    } else {
      const int before = t0 - (buf + GC) * BT;
      if (enter && before >= 0) load_dt(before);
      if (more) stage(t0 - BT);
    }
    const Gates<HALF>& g = sG[buf][hw];
    // The lane's addresses in the tiles, made anew for every chunk (the asm sees to
    // it): held over the loop they would spill.
    int lt = lane;
    asm volatile("" : "+v"(lt));
    const int rt = lt & 15, qt = lt >> 4;
    const int k_row = TK::row_at(rt, qt), m_row = TM::row_at(rt, qt);

    f32x4 Y[4][NB];
    if constexpr (OUT) {
      // ---- M: the wave's three of the 12 blocks of 16 x 16 on and under the
      // diagonal of 32 x 32 blocks, 3 w + i in the order (tb, sb) = (0, 0), (0, 1),
      // (1, 0), (1, 1), (2, 0) .. (2, 3), (3, 0) .. (3, 3)
      f32x4 E[3];
      int tbs[3], sbs[3];
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int n = 3 * w + i;
        tbs[i] = n < 4 ? n >> 1 : n < 8 ? 2 : 3;
        sbs[i] = n < 4 ? n & 1 : n & 3;
        E[i] = zero4();
      }
      auto score_frag = [&](const char* tile, int n, const int (&blk)[3]) {
        return TK::row_frag(tile, (k_row ^ (n / 3 * TK::slab_x)) + tiles::blk_rows(blk[n % 3]) * TK::row_bytes, 0);
      };
      Frag<T> bn = score_frag(sB, 0, sbs), cn = score_frag(sC, 0, tbs);
#pragma unroll
      for (int n = 0; n < 3 * KS; ++n) {
        const Frag<T> bf = bn, cf = cn;
        if (n + 1 < 3 * KS) {
          bn = score_frag(sB, n + 1, sbs);
          cn = score_frag(sC, n + 1, tbs);
          ahead();
        }
        E[n % 3] = mma(bf, cf, E[n % 3]);
      }
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        const int t = perm_row(0, rt) + tiles::blk_rows(tbs[i]);
        const int s0 = 8 * qt + tiles::blk_rows(sbs[i]);
        const int past = t - s0;   // slots above it are later tokens
#pragma unroll
        for (int hd = 0; hd < NH; ++hd) {
          const Gates<HALF>& gg = sG[buf][hd];
          const float gt = gg.g[t];
          const f32x4 ge = *reinterpret_cast<const f32x4*>(gg.e + s0);
          f32x4 M;
          if constexpr (HALF) {
#pragma unroll
            for (int e = 0; e < 4; ++e) M[e] = e <= past ? E[i][e] * ex2(gt - ge[e]) : 0.f;
          } else {
            const float gl = gg.lo[t];
            const f32x4 gs = *reinterpret_cast<const f32x4*>(gg.g + s0);
            const f32x4 gsl = *reinterpret_cast<const f32x4*>(gg.lo + s0);
#pragma unroll
            for (int e = 0; e < 4; ++e) M[e] = e <= past ? E[i][e] * ge[e] * ex2((gt - gs[e]) + (gl - gsl[e])) : 0.f;
          }
          // columns s0 .. s0 + 3 of row t
          char* mp = sM + hd * TM::bytes + (m_row ^ ((sbs[i] >> 1) * TM::slab_x)) + tiles::blk_rows(tbs[i]) * TM::row_bytes +
                     4 * (int)sizeof(T) * (sbs[i] & 1);
          const float m[4] = {M[0], M[1], M[2], M[3]};
          *reinterpret_cast<typename VecOf<4 * sizeof(T)>::type*>(mp) = pack(m, T());
        }
      }

      // ---- Y^T = 2^{G_t} S C^T
      Frag<T> cnext = TK::row_frag(sC, k_row, 0);
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
          const Frag<T> cf = cnext;
          if (4 * k + tb + 1 < 4 * KS) {
            cnext = TK::row_frag(sC, k_row ^ ((k + (tb + 1) / 4) * TK::slab_x), (tb + 1) % 4);
            ahead();
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) Y[tb][b] = mma(sf[b], cf, Y[tb][b]);
        }
      }
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const float eg = g.eg[perm_row(0, rt) + tiles::blk_rows(tb)];
#pragma unroll
        for (int b = 0; b < NB; ++b) Y[tb][b] *= eg;
      }
      tiles::lds_barrier();   // M is complete
    }

    // ---- Y^T += x^T M^T + D x^T
    const typename TX::Col x_col = TX::col_at(rt, qt, [&](int c) { return !OUT ? 4 * c : NB == 2 ? 32 * w + 8 * c : 16 * w + 4 * c; });
    const typename TK::Col b_col = TK::col_at(rt, qt, [&](int c) { return (OUT ? 8 : 4) * c; });
    const int p0 = 16 * NB * w + CL * qt;   // the lane's columns
    Frag<T> xf[2][NB];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int b = 0; b < NB; ++b) xf[j][b] = OUT ? TX::col_frag(sX, x_col, j, 0, b) : TX::col_blk(sX, x_col, j, NB * w + b);
    if constexpr (OUT) {
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
#pragma unroll
        for (int j = 0; j <= (tb >> 1); ++j) {
          const Frag<T> mf = TM::row_frag(sM + hw * TM::bytes, m_row ^ (j * TM::slab_x), tb);
#pragma unroll
          for (int b = 0; b < NB; ++b) Y[tb][b] = mma(xf[j][b], mf, Y[tb][b]);
        }
      }
      if (a.D) {
        const int x_row = TX::off(perm_row(0, rt), p0 * (int)sizeof(T) / 16) + (p0 * (int)sizeof(T) & 15);
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          const yvec xv = lds_vec<yvec>(sX + x_row + tiles::blk_rows(tb) * TX::row_bytes);
#pragma unroll
          for (int e = 0; e < CL; ++e) Y[tb][e >> 2][e & 3] = fmaf(skip, elem<T>(xv, e), Y[tb][e >> 2][e & 3]);
        }
      }
    }

    // ---- S <- 2^{G_63} S + (B^T) (w o x), in one or three bf16 terms of w o x
    const float dec = sDec[buf][hw];
    if constexpr (OUT) {
#pragma unroll
      for (int k = 0; k < KB; ++k)
#pragma unroll
        for (int b = 0; b < NB; ++b) S[k][b] *= dec;
    }
    auto update = [&](auto terms_) {
      constexpr int terms = decltype(terms_)::value;
      auto b_frag = [&](int j, int k) { return OUT ? TK::col_frag(sB, b_col, j, k >> 1, k & 1) : TK::col_blk(sB, b_col, j, k); };
      Frag<T> next = b_frag(0, 0);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Frag<T> xs[terms][NB];
        f32x4 v[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          v[h] = *reinterpret_cast<const f32x4*>(g.w + 32 * j + 8 * qt + 4 * h);
          if constexpr (!OUT) v[h] *= after;
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          f32x4 p[2];
#pragma unroll
          for (int e = 0; e < 8; ++e) p[e >> 2][e & 3] = xf[j][b].get(e) * v[e >> 2][e & 3];
#pragma unroll
          for (int m = 0; m < terms; ++m) {
            xs[m][b] = frag_of(p[0], p[1], T());
            if (m + 1 < terms) {
#pragma unroll
              for (int e = 0; e < 8; ++e) p[e >> 2][e & 3] -= xs[m][b].get(e);
            }
          }
        }
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          const Frag<T> bf = next;
          if (k + 1 < KB || j == 0) {
            next = b_frag(k + 1 < KB ? j : 1, k + 1 < KB ? k + 1 : 0);
            ahead();
          }
#pragma unroll
          for (int m = 0; m < terms; ++m)
#pragma unroll
            for (int b = 0; b < NB; ++b) S[k][b] = mma(bf, xs[m][b], S[k][b]);
        }
      }
    };
    if (HALF && fine) update(tiles::Int<HALF ? 3 : 1>{});
    else update(tiles::Int<1>{});
    if constexpr (!OUT) after *= dec;
    int le = lane;
    asm volatile("" : "+v"(le));
    const int t_row = perm_row(0, le & 15);            // y and z: rows t_row + blk_rows(tb)
    const uint32_t col_b = (16 * NB * w + CL * (le >> 4)) * (uint32_t)sizeof(T);
    yvec zr[4];   // not with the tiles: registers that the products need
    if (OUT && a.z.p) {
#pragma unroll
      for (int tb = 0; tb < 4; ++tb) {
        const char* zt = wz.at(t0 + tiles::blk_rows(tb));
        if (t_row + tiles::blk_rows(tb) < nr) zr[tb] = gload<yvec>(zt + ((uint32_t)t_row * wz.stride + col_b));
      }
    }
    if constexpr (OUT) wait_vm<0>();   // z: behind the next tiles' loads the compiler would wait for those too
    tiles::lds_barrier();   // everyone is done with the tiles
    if constexpr (OUT) {
      // ---- y, gated
      const char* const yc = wy.at(t0);
      auto finish = [&](auto full_) {
#pragma unroll
        for (int tb = 0; tb < 4; ++tb) {
          float y[CL];
#pragma unroll
          for (int e = 0; e < CL; ++e) y[e] = Y[tb][e >> 2][e & 3];
          if (a.z.p) {
#pragma unroll
            for (int e = 0; e < CL; ++e) {
              const float ze = elem<T>(zr[tb], e);
              y[e] *= ze * __builtin_amdgcn_rcpf(1.0f + __expf(-ze));
            }
          }
          char* yt = const_cast<char*>(yc) + (uint64_t)wy.stride * (uint32_t)tiles::blk_rows(tb);
          asm volatile("" : "+s"(yt));
          if (decltype(full_)::value || t_row + tiles::blk_rows(tb) < nr)
            gstore<yvec>(yt + ((uint32_t)t_row * wy.stride + col_b), pack(y, T()));
        }
      };
      if (!more) {
        finish(tiles::Int<0>{});
        break;
      }
      load_tiles(t0 + BT);
      asm volatile("" ::: "memory");   // the stores stay behind the loads
      finish(tiles::Int<1>{});
    }
  }

  // ---- the final state
  if (!OUT || out_ht) {
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      float* p = (OUT ? a.ht : seg_state) + state_at(OUT ? sg.n : sg.state, b);
#pragma unroll
      for (int k = 0; k < KB; ++k)
        *reinterpret_cast<f32x4*>(p + (OUT ? 32 * (k >> 1) + 4 * (k & 1) : 16 * k)) = S[k][b];
    }
  }
  if constexpr (!OUT) {   // the waves' shares of the log-decay, in order
    tiles::lds_barrier();
    if (tid < NH) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < GC; ++i) sum += sSum[i * NH + tid];
      seg_decay[(size_t)sg.state * a.HV + hv0 + tid] = sum;
    }
  }
}

// Joins the segments of a split call: each segment's own final state (from zeros)
// becomes the state behind it, in place; the last one's is ht (its slot holds
// nothing where ht is not asked for).
// A thread owns four elements of a (sequence, head) and walks down its segments,
// the loads of four in flight together.  Memory-bound: every state once in and out
// (16 segments x 64 heads of 64 x 128: 67 MB in 12.5 us, 5.4 TB/s).  Each segment's
// work-groups joining what lies before them instead, in the last launch, took 5 us
// off 5 segments a prompt and added 37 to 16 (their reads are serial and repeated).
__global__ __launch_bounds__(256) void ssm_join_kernel(SsmArgs a, int seg, int states, int blocks_per_head,
                                                       float* __restrict__ seg_state,
                                                       const double* __restrict__ seg_decay,
                                                       SplitSeq* __restrict__ table) {
  const int lane = threadIdx.x & 63;
  const int mh = blockIdx.x / blocks_per_head;
  const int part = blockIdx.x - mh * blocks_per_head;
  const int m = mh / a.HV, hv = mh - m * a.HV;   // the m-th sequence of those that are split
  int n = m, slot0 = 0, segs = 1;
  if (!a.cu) {
    segs = a.T > seg ? (a.T + seg - 1) / seg : 1;
    slot0 = n * segs;
  } else {
    int before = 0;   // split sequences before these 64
    n = -1;
    for (int base = 0; base < a.N; base += 64) {
      const int st = states_of(a, seg, base + lane);
      const LaneSum sum(st, lane);
      const unsigned long long cut = __ballot(st > 0);
      if (m < before + __popcll(cut)) {
        const int rank = before + __popcll(cut & ((1ULL << lane) - 1));
        const int l = __ffsll((unsigned long long)__ballot(st > 0 && rank == m)) - 1;
        n = base + l;
        segs = __builtin_amdgcn_readlane(st, l);
        slot0 += __builtin_amdgcn_readlane(sum.incl, l) - segs;
        break;
      }
      before += __popcll(cut);
      slot0 += sum.all;
    }
    // boundaries out of order may claim more states than there are
    if (n < 0 || slot0 < 0 || slot0 >= states) segs = 0;
    else if (segs > states - slot0) segs = states - slot0;
    if (hv == 0 && part == 0 && threadIdx.x == 0) table[m] = SplitSeq{n, slot0, segs, 0};
  }
  if (segs < 2) return;
  const int own_states = segs - (a.ht ? 0 : 1);
  const size_t VK = (size_t)a.V * a.K, head = (size_t)a.HV * VK;
  const size_t e0 = ((size_t)part * 256 + threadIdx.x) * 4;
  f32x4 st = zero4();
  if (a.h0) st = *reinterpret_cast<const f32x4*>(a.h0 + (size_t)n * head + hv * VK + e0);
  float* p = seg_state + (size_t)slot0 * head + hv * VK + e0;
  // the decays by vector loads: as scalar ones they hold up the loop (13.6 us in place of 12.5 above)
  int slot_v = slot0;
  asm("" : "+v"(slot_v));
  const double* d = seg_decay + (size_t)slot_v * a.HV + hv;
  constexpr int U = 4;
  for (int j = 0; j < own_states; j += U) {
    f32x4 own[U];
    float f[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = j + u < own_states ? j + u : j;
      own[u] = *reinterpret_cast<const f32x4*>(p + i * head);
      f[u] = ex2((float)d[(size_t)i * a.HV]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + u < own_states) {
#pragma unroll
        for (int e = 0; e < 4; ++e) st[e] = fmaf(f[u], st[e], own[u][e]);
        if (j + u < segs - 1) *reinterpret_cast<f32x4*>(p + (size_t)(j + u) * head) = st;
      }
    }
  }
  if (a.ht) *reinterpret_cast<f32x4*>(a.ht + (size_t)n * head + hv * VK + e0) = st;
}

template <typename T, int K, int V, int NH>
hipError_t launch_t(const SsmArgs& a, const SsmPlan& p, hipStream_t s) {
  const int tiles = a.HV / NH;
  auto grid = [&](int slots) { return dim3((unsigned)((slots * tiles + 7) / 8 * 8)); };
  float* st = reinterpret_cast<float*>(a.workspace);
  char* const ws = reinterpret_cast<char*>(a.workspace);
  double* dec = p.split ? reinterpret_cast<double*>(ws + p.decay_off) : nullptr;
  SplitSeq* table = p.split ? reinterpret_cast<SplitSeq*>(ws + p.table_off) : nullptr;
  if (p.split) {
    hipLaunchKernelGGL((ssm_scan_kernel<T, K, V, NH, false>), grid(p.states), dim3(64 * NW), 0, s, a, p.seg, p.slots,
                       p.states, true, table, 0, st, dec);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    constexpr int per_head = K * V / 1024;
    hipLaunchKernelGGL(ssm_join_kernel, dim3((unsigned)((long long)p.joins * a.HV * per_head)), dim3(256), 0, s, a,
                       p.seg, p.states, per_head, st, dec, table);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL((ssm_scan_kernel<T, K, V, NH, true>), grid(p.slots), dim3(64 * NW), 0, s, a, p.seg, p.slots,
                     p.states, p.split, table, p.joins, st, dec);
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
  // One round of work-groups on 256 CUs: two a CU, one with fp32 tiles (bf16, one
  // prompt of 8192 tokens x 64 heads: 256 work-groups 148 us, 512 117, 768 144, 1024
  // 140; fp32, 4096 tokens x 32 heads: 128 195, 256 116, 512 123).  But no segment shorter than 2 sqrt(T) tokens: halving the segments
  // saves two launches the half of their chunks and costs the join as many steps
  // (2048 tokens x 32 heads: 64-token segments 41 us, 128 37, 256 47; 700 x 16
  // heads: 64 25, 128 28, 256 40).
  const long long want = bf16 ? 512 : 256;
  // packed sequences end in half a segment on average, up to half of the work-groups
  const long long tails = !varlen ? 0 : tiles * N < want ? tiles * N / 2 : want / 2;
  long long seg = ((tokens * tiles + want - tails - 1) / (want - tails) + 63) / 64 * 64;
  const long long least = ((long long)(2.0 * sqrt((double)T)) + 63) / 64 * 64;
  seg = seg < least ? least : seg;
  // nor two chunks alone: they cost less than two more launches (128 tokens x 8 heads
  // 16.1 us in one launch, 18.7 in three; 192 tokens 21.7 and 19.2)
  // nor so many sequences that the first launch's look at their boundaries is what counts
  const bool join = (long long)N * HV * (K * V / 1024) < (1 << 24);
  if (seg >= T || T <= 128 || !join) seg = ((long long)T + 63) / 64 * 64;
  p.split = seg < T;
  p.seg = seg > 64 ? (int)seg : 64;
  p.slots = !p.split ? N : (varlen ? (int)(tokens / seg) + N : N * (int)((T + seg - 1) / seg));
  // A packed sequence that is split has seg + 1 tokens or more, and of n such with L
  // tokens in all the sum of ceil(length / seg) is at most (L - n) / seg + n.
  const long long most = p.split && varlen ? tokens / (seg + 1) : N;
  p.joins = (int)(most < N ? most : N);
  p.states = !p.split || !varlen ? p.slots : (int)((tokens - p.joins) / seg) + p.joins;
  const size_t state = (size_t)p.states * HV * V * K * 4;
  p.decay_off = (state + 255) / 256 * 256;
  p.table_off = p.decay_off + ((size_t)p.states * HV * 8 + 255) / 256 * 256;
  p.bytes = p.split ? p.table_off + (varlen ? ((size_t)p.joins * sizeof(SplitSeq) + 255) / 256 * 256 : 0) : 0;
  return p;
}

hipError_t launch_ssm_fwd(const SsmArgs& a, hipStream_t s) {
  const SsmPlan p = ssm_plan(a.nb, a.T, a.Hk, a.HV, a.K, a.V, a.N, a.cu != nullptr, a.bf16 != 0);
  return a.bf16 ? launch_io<bf16_t>(a, p, s) : launch_io<float>(a, p, s);
}

}  // namespace gdn
