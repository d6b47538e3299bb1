// Gradients of the chunked gated delta rule (scalar gate): the arrays that pass
// between its launches, and what the kernels share.  Per chunk of 64 tokens, with
// G the chunk-local cumulative gate, h = S^T [K, V] at the chunk's start, dh' the
// gradient of the state at its end, A = (I + L)^-1 and P = scale tril(Q K^T o Gamma)
// of the prefill's intra step:
//
//   states      R = beta (V - e^G K h),  Vn = A R,
//               h <- e^{G_last} h + (e^{G_last - G} K)^T Vn
//   gradients   Y = P^T dO + e^{G_last - G} K dh',  dR = A^T Y,
//               dh <- e^{G_last} dh' + scale (e^G Q)^T dO - (beta e^G K)^T dR
//   then        dq = scale (e^G dO h^T + tril(dO Vn^T o Gamma) K)
//               E  = -(e^G dR h^T + stril(dR Vn^T o Gamma) K)
//               W  = e^{G_last - G} Vn dh'^T + scale tril(dO Vn^T o Gamma)^T Q
//                    - stril(dR Vn^T o Gamma)^T (beta K)
//               dk = beta E + W,  dv = beta dR,  dbeta = v . dR + k . E
//               dG = q . dq + beta k . E - k . W;  at the chunk's last row also
//               <h', dh'> = e^{G_last} <h, dh'> + sum_t k_t . (e^{G_last - G_t} dh' Vn_t);
//               dg = the sums of dG from each row to the chunk's end
//
// Every array that holds a gradient is kept times a power of two, one for each
// (sequence, key head), that brings the largest of its dO and dht to 2 .. 4: with
// bf16 io the operands of the products are fp16 (2^-11 where bf16 has 2^-8), and
// the gradients of a mean over many tokens lie far below fp16's normal numbers.  Rows
// that enter a product times their tokens' gate factor are rounded three times: the row,
// the factor, their product.  (The prefill carries its state's operands as pairs of fp16;
// here they are single ones, and the state that is differentiated around is that.)
#pragma once

#include "gdn_device.h"
#include "gdn_launch.h"
#include "scan_tiles.h"

namespace gdn {
namespace bwd {

constexpr int BT = 64;
using tiles::perm_row;

// The power of two that brings `amax` to 2 .. 4 (and its inverse); NaN where it is
// not finite, which then every gradient of the (sequence, key head) becomes.
__device__ __forceinline__ float grad_scale(uint32_t amax_bits, float& inverse) {
  const int e = (int)(amax_bits >> 23);   // biased exponent; the sign is clear
  int up = amax_bits == 0 ? 0 : 128 - e;  // 2^up amax in [2, 4)
  up = up > 126 ? 126 : up < -126 ? -126 : up;
  float s = __builtin_bit_cast(float, (uint32_t)(127 + up) << 23);
  inverse = __builtin_bit_cast(float, (uint32_t)(127 - up) << 23);
  if (e == 255) s = inverse = __builtin_bit_cast(float, 0x7FC00000u);
  return s;
}

// Eight values in a row from the two accumulators that hold them.
__device__ __forceinline__ f32x8 both(const f32x4& a, const f32x4& b) {
  return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Hides where a value comes from: offsets made from it are made where they are used, a
// cheap operation each, instead of once in front of all loops, which takes more registers
// than there are.
template <typename I>
__device__ __forceinline__ I opaque(I x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Two accumulators as one operand fragment.  fp16 without saturation: a value past
// 65504 becomes an infinity, which shows in the result.
__device__ __forceinline__ void join(Frag<f16_t>& f, const f32x4& a, const f32x4& b) {
  f.v = __builtin_convertvector(both(a, b), f16x8);
}
__device__ __forceinline__ void join(Frag<float>& f, const f32x4& a, const f32x4& b) {
  f.v = both(a, b);
}

// Eight consecutive values of the io type as the compute type.
__device__ __forceinline__ Frag<f16_t> widen(const Frag<bf16_t>& a, float s) {
  Frag<f16_t> r;
  r.v = __builtin_convertvector(__builtin_convertvector(a.v, f32x8) * s, f16x8);
  return r;
}
__device__ __forceinline__ Frag<f16_t> widen(const Frag<bf16_t>& a) {
  Frag<f16_t> r;
  r.v = __builtin_convertvector(__builtin_convertvector(a.v, f32x8), f16x8);
  return r;
}
__device__ __forceinline__ Frag<float> widen(const Frag<float>& a, float s) {
  Frag<float> r;
  r.v = a.v * s;
  return r;
}
__device__ __forceinline__ Frag<float> widen(const Frag<float>& a) { return a; }

// ... times a factor (fp16: one more rounding of each)
__device__ __forceinline__ Frag<f16_t> times(const Frag<f16_t>& a, float s) {
  Frag<f16_t> r;
  r.v = a.v * (_Float16)s;
  return r;
}
__device__ __forceinline__ Frag<float> times(const Frag<float>& a, float s) {
  Frag<float> r;
  r.v = a.v * s;
  return r;
}

__device__ __forceinline__ f32x8 values(const Frag<f16_t>& a) { return __builtin_convertvector(a.v, f32x8); }
__device__ __forceinline__ f32x8 values(const Frag<float>& a) { return a.v; }
__device__ __forceinline__ f32x8 values(const Frag<bf16_t>& a) { return __builtin_convertvector(a.v, f32x8); }

__device__ __forceinline__ void store8(f16_t* p, const Frag<f16_t>& f) {
  store_nt16(p, __builtin_bit_cast(tiles::u32x4, f.v));
}
__device__ __forceinline__ void store8(float* p, const Frag<float>& f) {
  store_nt16(p, f32x4{f.v[0], f.v[1], f.v[2], f.v[3]});
  store_nt16(p + 4, f32x4{f.v[4], f.v[5], f.v[6], f.v[7]});
}
// ... eight fp32 values in the io type.  Not as streaming stores: the waves of a
// work-group write the halves of a line, which the L2 joins.
__device__ __forceinline__ void store_io8(bf16_t* p, const f32x8& x) {
  *reinterpret_cast<tiles::u32x4*>(p) =
      tiles::u32x4{pack_bf2(x[0], x[1]), pack_bf2(x[2], x[3]), pack_bf2(x[4], x[5]), pack_bf2(x[6], x[7])};
}
__device__ __forceinline__ void store_io8(float* p, const f32x8& x) {
  *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4*>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}

// An LDS tile of rows of COLS elements.  16-bit: 16-byte units swizzled by row as
// in the prefill's scan (row fragments and transposing reads without bank
// conflicts).  fp32: rows padded by 16 bytes.
//
// A lane's fragments lie at one offset each for a set of them (rows(), cols()) plus
// constants: the swizzle of a row does not change with the 4 and 32 rows that
// separate them.
template <typename C, int COLS> struct Tile;
template <int COLS> struct Tile<f16_t, COLS> {
  static constexpr int pitch = 2 * COLS;
  static constexpr int odd = 8;   // from block 2 m of a permuted pair to block 2 m + 1
  static constexpr int bytes(int rows) { return rows * pitch; }
  static __device__ __forceinline__ int off(int row, int col) {   // byte of an element; col a multiple of 4
    int u;
    if constexpr (COLS == 128) u = tiles::qk_off<128>(row, col >> 3);
    else u = tiles::a_off(row, col >> 3);
    return u + 2 * (col & 4);
  }
  static __device__ __forceinline__ void put(char* t, int row, int col, const Frag<f16_t>& f) {
    *reinterpret_cast<f16x8*>(t + off(row, col)) = f.v;
  }
  // four consecutive values of a row
  static __device__ __forceinline__ void put4(char* t, int row, int col, const f32x4& x) {
    typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<f16x4*>(t + off(row, col)) = __builtin_convertvector(x, f16x4);
  }
  static __device__ __forceinline__ Frag<f16_t> row(const char* t) {   // 8 values of a row
    Frag<f16_t> f;
    f.v = *reinterpret_cast<const f16x8*>(t);
    return f;
  }
  static __device__ __forceinline__ Frag<f16_t> row8(const char* t, int r, int col) { return row(t + off(r, col)); }
  // offset of rows 8 g .. 8 g + 7 of the lane's column: column 32 pair + perm_row(0, n), or 16 blk + n
  static __device__ __forceinline__ int pair_cols(int pair, int n, int g) {
    return off(8 * g + (n >> 2), 32 * pair + 8 * (n & 3));
  }
  static __device__ __forceinline__ int block_cols(int blk, int n, int g) {
    return off(8 * g + (n >> 2), 16 * blk + 4 * (n & 3));
  }
  // from the offset of block 0 to that of block b of the columns, of 16 rows b and 32-column slab s (of 64 columns)
  static __device__ __forceinline__ int to_block(int o, int b) { return o ^ (b << 5); }
  static __device__ __forceinline__ int to_rows(int o, int b, int s = 0) {
    return (o ^ (((b & 1) << 5) | (s << 6))) + b * 16 * pitch;
  }
  static __device__ __forceinline__ Frag<f16_t> col(const char* t) {   // 8 values of a column, by transposing reads
    const uint2 lo = tiles::ld_tr(t), hi = tiles::ld_tr(t + 4 * pitch);
    Frag<f16_t> f;
    f.v = __builtin_bit_cast(f16x8, tiles::u32x4{lo.x, lo.y, hi.x, hi.y});
    return f;
  }
};
template <int COLS> struct Tile<float, COLS> {
  static constexpr int pitch = 4 * COLS + 16;
  static constexpr int odd = 16;
  static constexpr int bytes(int rows) { return rows * pitch; }
  static __device__ __forceinline__ int off(int row, int col) { return row * pitch + 4 * col; }
  static __device__ __forceinline__ void put(char* t, int row, int col, const Frag<float>& f) {
    float* p = reinterpret_cast<float*>(t + off(row, col));
    *reinterpret_cast<f32x4*>(p) = f32x4{f.v[0], f.v[1], f.v[2], f.v[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{f.v[4], f.v[5], f.v[6], f.v[7]};
  }
  static __device__ __forceinline__ void put4(char* t, int row, int col, const f32x4& x) {
    *reinterpret_cast<f32x4*>(t + off(row, col)) = x;
  }
  static __device__ __forceinline__ Frag<float> row(const char* t) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(t), b = *reinterpret_cast<const f32x4*>(t + 16);
    Frag<float> f;
    f.v = both(a, b);
    return f;
  }
  static __device__ __forceinline__ Frag<float> row8(const char* t, int r, int col) { return row(t + off(r, col)); }
  static __device__ __forceinline__ int pair_cols(int pair, int n, int g) { return off(8 * g, 32 * pair + perm_row(0, n)); }
  static __device__ __forceinline__ int block_cols(int blk, int n, int g) { return off(8 * g, 16 * blk + n); }
  static __device__ __forceinline__ int to_block(int o, int b) { return o + 64 * b; }
  static __device__ __forceinline__ int to_rows(int o, int b, int s = 0) { return o + b * 16 * pitch + 128 * s; }
  static __device__ __forceinline__ Frag<float> col(const char* t) {
    Frag<float> f;
#pragma unroll
    for (int e = 0; e < 8; ++e) f.v[e] = *reinterpret_cast<const float*>(t + e * pitch);
    return f;
  }
};

// [rows of V][COLS] arrays that the scans leave for the chunks' gradients (h, dh': COLS =
// K; Vn^T, dR^T: 64 tokens), in memory and, 32 rows at a time, in LDS alike.  fp16: for 16
// rows and 32 columns one piece of 1 KiB, which a wave stores in one go: the 16 bytes
// (columns 8 g .. 8 g + 7) of row n at unit 16 g + (n ^ 4 g).  That order, copied as it is,
// leaves the transposing reads without bank conflicts.  fp32: rows.
template <typename C, int COLS> struct Kept;
template <int COLS> struct Kept<f16_t, COLS> {
  static constexpr int odd = 8;
  static constexpr int bytes = 32 * COLS * 2;   // of 32 rows
  // element of the 8 columns 32 s + 8 g of row 16 blk + n
  static __device__ __forceinline__ uint32_t at(int blk, int s, int n, int g) {
    return (uint32_t)((blk * (COLS / 32) + s) * 64 + g * 16 + (n ^ 4 * g)) * 8;
  }
  // as in Tile: columns of block pair `pair` in the permuted order, of 16-column block 0, of block b
  static __device__ __forceinline__ int pair_cols(int pair, int n, int g) {
    return ((g >> 1) * (COLS / 32) + pair) * 1024 + (n & 3) * 256 + ((8 * (g & 1) + (n >> 2)) ^ 4 * (n & 3)) * 16;
  }
  static __device__ __forceinline__ int block_cols(int n, int g) {
    const int u = (n & 3) >> 1;
    return (g >> 1) * (COLS / 32) * 1024 + u * 256 + ((8 * (g & 1) + (n >> 2)) ^ 4 * u) * 16 + (n & 1) * 8;
  }
  static __device__ __forceinline__ int to_block(int o, int b) { return (o ^ (b & 1) * 128) + (b & 1) * 512 + (b >> 1) * 1024; }
  static __device__ __forceinline__ Frag<f16_t> col(const char* t, int o) {   // rows four on: the other bit of the unit
    const uint2 lo = tiles::ld_tr(t + o), hi = tiles::ld_tr(t + (o ^ 64));
    Frag<f16_t> f;
    f.v = __builtin_bit_cast(f16x8, tiles::u32x4{lo.x, lo.y, hi.x, hi.y});
    return f;
  }
};
template <int COLS> struct Kept<float, COLS> {
  typedef Tile<float, COLS> L;
  static constexpr int odd = L::odd;
  static constexpr int bytes = L::bytes(32);
  static __device__ __forceinline__ uint32_t at(int blk, int s, int n, int g) {
    return (uint32_t)((16 * blk + n) * COLS + 32 * s + 8 * g);
  }
  static __device__ __forceinline__ int pair_cols(int pair, int n, int g) { return L::pair_cols(pair, n, g); }
  static __device__ __forceinline__ int block_cols(int n, int g) { return L::block_cols(0, n, g); }
  static __device__ __forceinline__ int to_block(int o, int b) { return L::to_block(o, b); }
  static __device__ __forceinline__ Frag<float> col(const char* t, int o) { return L::col(t + o); }
};

}  // namespace bwd
}  // namespace gdn
