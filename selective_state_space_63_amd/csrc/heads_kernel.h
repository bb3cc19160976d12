// heads_kernel.h -- building blocks of the multi-head scan's matrix-core
// kernels: operand fragments, LDS tiles and the steps of a chunk.
//
// Matrix products are 16 x 16 tiles with K = 32 per step: lane 16 g + c holds
// the 8 K-values of row (or column) c that belong to lane group g, and the
// result's rows 4 g .. 4 g + 3 of column c.  Which 8 of the 32 K-values a
// group holds is free as long as both operands agree; here group g holds
//   k = 4 g .. 4 g + 3 and 16 + 4 g .. 16 + 4 g + 3,
// which is what two stacked results (rows 0-15 and 16-31) hold per lane.  So a
// result -- a tile of the state, or of the decayed Gram matrix -- becomes an
// operand of the next product in registers, without a shuffle.
//
// LDS tiles come in two layouts, both without padding.  RowTile, for operands
// along its rows: the columns of each 32 lie in the order of K above (chunks of
// four: 0, 4, 1, 5, 2, 6, 3, 7), so an operand is one 16-byte read per lane.
// ColTile, for operands down its columns (read with the transposing LDS read:
// 16 lanes fetch 32 bytes of each of four rows): columns in order.  The
// 16-byte (RowTile) or 32-byte units of a row are XORed with bits of the row
// so that no read meets a bank twice.  Measured with SQ_LDS_BANK_CONFLICT on
// each access alone (cycles per instruction, bf16): a 16-byte read takes 4
// when lanes 0-3, 12-15, 20-27 cover all 64 banks (and the three like sets),
// an 8-byte or transposing read 2 when lanes 0-31 do; writes take 16 lanes of
// 8 bytes or 8 of 16 over 32 banks per cycle.
//
// bf16: one 16 x 16 x 32 matrix instruction.  fp32: eight 16 x 16 x 4 ones.
#ifndef S6_HEADS_KERNEL_H_
#define S6_HEADS_KERNEL_H_

#include "block_internal.h"

namespace s6i {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kTP = 64;      // channels of a head per workgroup (a wider head is several tiles)
constexpr int kHQ = 64;      // tokens per chunk of the scan

template <typename In>
struct Frag;
template <>
struct Frag<uint16_t> {
  bf16x8 v;
};
template <>
struct Frag<float> {
  float v[8];
};

__device__ __forceinline__ f32x4 mma(const Frag<uint16_t>& a, const Frag<uint16_t>& b, f32x4 d) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a.v, b.v, d, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mma(const Frag<float>& a, const Frag<float>& b, f32x4 d) {
#pragma unroll
  for (int j = 0; j < 8; ++j) d = __builtin_amdgcn_mfma_f32_16x16x4f32(a.v[j], b.v[j], d, 0, 0, 0);
  return d;
}

__device__ __forceinline__ float frag_f32(const Frag<uint16_t>& f, int j) { return (float)f.v[j]; }
__device__ __forceinline__ float frag_f32(const Frag<float>& f, int j) { return f.v[j]; }

// Eight floats as an operand (bf16: rounded to nearest even).
__device__ __forceinline__ void to_frag(const float (&f)[8], Frag<uint16_t>& o) {
#pragma unroll
  for (int j = 0; j < 8; ++j) o.v[j] = (__bf16)f[j];
}
__device__ __forceinline__ void to_frag(const float (&f)[8], Frag<float>& o) {
#pragma unroll
  for (int j = 0; j < 8; ++j) o.v[j] = f[j];
}

// Eight floats as the sum of two operands: bf16 parts (the first rounded to
// nearest, the second the rounded rest: within 2^-17), or the floats and
// nothing.
template <typename In>
struct Pair {
  Frag<In> hi, lo;
};
// The rests of two floats after their packed bf16 parts; the parts as an
// operand.  (Two values at a time: the compiler converts a value that is also
// read back as a float by itself, and once more to pack it.)
__device__ __forceinline__ uint32_t split2(float& a, float& b) {
  uint32_t p = bf_pack(a, b);
  asm("" : "+v"(p));
  a -= bf_low(p);
  b -= bf_high(p);
  return p;
}
typedef unsigned int gu32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ void to_pair(const float (&f)[8], Pair<uint16_t>& o) {
  gu32x4 hi, lo;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = f[2 * j], b = f[2 * j + 1];
    hi[j] = split2(a, b);
    lo[j] = bf_pack(a, b);
  }
  o.hi.v = __builtin_bit_cast(bf16x8, hi);
  o.lo.v = __builtin_bit_cast(bf16x8, lo);
}
__device__ __forceinline__ void to_pair(const float (&f)[8], Pair<float>& o) { to_frag(f, o.hi); }

// d += (hi + lo) b
__device__ __forceinline__ f32x4 mma_pair(const Pair<uint16_t>& a, const Frag<uint16_t>& b, f32x4 d) {
  return mma(a.lo, b, mma(a.hi, b, d));
}
__device__ __forceinline__ f32x4 mma_pair(const Pair<float>& a, const Frag<float>& b, f32x4 d) { return mma(a.hi, b, d); }
// d += a (hi + lo)
__device__ __forceinline__ f32x4 mma_pair(const Frag<uint16_t>& a, const Pair<uint16_t>& b, f32x4 d) {
  return mma(a, b.lo, mma(a, b.hi, d));
}
__device__ __forceinline__ f32x4 mma_pair(const Frag<float>& a, const Pair<float>& b, f32x4 d) { return mma(a, b.hi, d); }

// Eight floats as the exact sum of operands: three bf16 parts hold the 24 bits
// of a float (down to the smallest bf16), one float part itself.  For what
// the state keeps: two parts would leave 2^-17 of every term in it.
template <typename In>
struct Whole {
  static constexpr int kParts = sizeof(In) == 2 ? 3 : 1;
  Frag<In> part[kParts];
};
__device__ __forceinline__ void to_whole(const float (&f)[8], Whole<uint16_t>& o) {
  gu32x4 w[3];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a = f[2 * j], b = f[2 * j + 1];
    w[0][j] = split2(a, b);
    w[1][j] = split2(a, b);
    w[2][j] = bf_pack(a, b);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) o.part[i].v = __builtin_bit_cast(bf16x8, w[i]);
}
__device__ __forceinline__ void to_whole(const float (&f)[8], Whole<float>& o) { to_frag(f, o.part[0]); }
// d += a b, the smallest parts first
template <typename In>
__device__ __forceinline__ f32x4 mma_whole(const Whole<In>& a, const Frag<In>& b, f32x4 d) {
#pragma unroll
  for (int i = Whole<In>::kParts - 1; i >= 0; --i) d = mma(a.part[i], b, d);
  return d;
}

// ------------------------------------------------------------- LDS tiles --
// Eight consecutive values of LDS as an operand.
__device__ __forceinline__ Frag<uint16_t> eight(const uint16_t* p) {
  Frag<uint16_t> o;
  o.v = *reinterpret_cast<const bf16x8*>(p);
  return o;
}
__device__ __forceinline__ Frag<float> eight(const float* p) {
  Frag<float> o;
  load_vec<float, 8>(p, o.v);
  return o;
}
// Four and four.
__device__ __forceinline__ Frag<uint16_t> four_four(const uint16_t* p, const uint16_t* q) {
  const s16x4 a = *reinterpret_cast<const s16x4*>(p), b = *reinterpret_cast<const s16x4*>(q);
  Frag<uint16_t> o;
  o.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  return o;
}
__device__ __forceinline__ Frag<float> four_four(const float* p, const float* q) {
  Frag<float> o;
  float a[4], b[4];
  load_vec<float, 4>(p, a);
  load_vec<float, 4>(q, b);
#pragma unroll
  for (int j = 0; j < 4; ++j) { o.v[j] = a[j]; o.v[4 + j] = b[j]; }
  return o;
}
// Rows r0 .. r0 + 3 and r0 + 16 .. r0 + 19 (r0 = 4 g of the group) of one column.
// bf16: the transposing read gives each lane four rows of its column, from
// 8-byte chunks that the 16 lanes of a group fetch (lane c: row c / 4 of the
// four, chunk c % 4 of the sixteen columns); `p` is the lane's chunk, `d` the
// distance of 16 rows.
__device__ __forceinline__ Frag<uint16_t> tr_read(const uint16_t* p, int d) {
  typedef __attribute__((address_space(3))) s16x4* lds4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uint16_t*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uint16_t*)(p + d));
  Frag<uint16_t> o;
  o.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  return o;
}

// A tile of COLS columns, for operands along its rows.  An address is a
// lane's part XORed with the unit; `lane` below is that part.
template <typename In, int COLS>
struct RowTile {
  static constexpr int size(int rows) { return rows * COLS; }
  static constexpr int kU = COLS / 8;  // units of 8 columns
  static_assert(kU == 4 || kU == 8 || kU == 16, "the rows' XOR");
  In* t;
  static __device__ __forceinline__ int mix(int row) {
    if constexpr (kU == 16) return row & 15;
    if constexpr (kU == 8) return ((row >> 1) & 7) ^ (row & 1);
    // 0, 2, 3, 1: two neighbours' units and the other two's, XORed with 1, are all four
    return ((row >> 2) & 1) * 2 ^ ((row >> 3) & 1) * 3;
  }
  // chunk m: columns 4 m .. 4 m + 3
  static __device__ __forceinline__ int at(int row, int m) {
    return row * COLS + 8 * ((((m & ~7) >> 1) + (m & 3)) ^ mix(row)) + 4 * ((m >> 2) & 1);
  }
  static __device__ __forceinline__ int row_lane(int g, int c) { return c * COLS + 8 * (g ^ mix(c)); }
  // K = columns 32 kk .. + 31 of row r + c (r a multiple of 16)
  __device__ __forceinline__ Frag<In> row(int lane, int r, int kk) const {
    return eight(t + (lane ^ (32 * kk)) + r * COLS);
  }
  // K = rows 32 kk .. + 31 of column 16 q + c
  __device__ __forceinline__ Frag<In> col(int q, int kk, int g, int c) const {
    if constexpr (sizeof(In) == 2) {
      return tr_read(t + at(4 * g + (c >> 2), 4 * q + (c & 3)) + 32 * kk * COLS, 16 * COLS);
    } else {
      Frag<In> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const In* p = t + at(32 * kk + 4 * g + j, 4 * q + (c >> 2)) + (c & 3);
        o.v[j] = p[0];
        o.v[4 + j] = p[16 * COLS];
      }
      return o;
    }
  }
  // columns 4 m .. 4 m + 3 of a row as floats
  __device__ __forceinline__ void four(int r, int m, float (&f)[4]) const { load_vec<In, 4>(t + at(r, m), f); }
};

// A tile of COLS columns, for operands down its columns.
template <typename In, int COLS>
struct ColTile {
  static constexpr int size(int rows) { return rows * COLS; }
  In* t;
  static __device__ __forceinline__ int mix(int row) {  // of the units of 16 columns
    return COLS >= 128 ? row & 7 : COLS >= 64 ? (row >> 1) & 3 : (row >> 2) & 1;
  }
  static __device__ __forceinline__ int at(int row, int m) {
    return row * COLS + 16 * ((m >> 2) ^ mix(row)) + 4 * ((m & 3) ^ (2 * ((row >> 3) & 1)));
  }
  static __device__ __forceinline__ int row_lane(int g, int c) { return at(c, g); }
  static __device__ __forceinline__ int col_lane(int g, int c) { return at(4 * g + (c >> 2), c & 3); }
  // K = columns 32 kk .. + 31 of row r + c (r a multiple of 16)
  __device__ __forceinline__ Frag<In> row(int lane, int r, int kk) const {
    return four_four(t + (lane ^ (32 * kk)) + r * COLS, t + (lane ^ (32 * kk + 16)) + r * COLS);
  }
  // K = rows 32 kk .. + 31 of column 16 q + c
  __device__ __forceinline__ Frag<In> col(int lane, int q, int kk, int g, int c) const {
    if constexpr (sizeof(In) == 2) {
      return tr_read(t + (lane ^ (16 * q)) + 32 * kk * COLS, 16 * COLS);
    } else {
      Frag<In> o;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const In* p = t + at(32 * kk + 4 * g + j, 4 * q + (c >> 2)) + (c & 3);
        o.v[j] = p[0];
        o.v[4 + j] = p[16 * COLS];
      }
      return o;
    }
  }
  __device__ __forceinline__ void four(int r, int m, float (&f)[4]) const { load_vec<In, 4>(t + at(r, m), f); }
};

// An operand kept in LDS as such: 8 values per lane.
template <typename In>
__device__ __forceinline__ Frag<In> lane_frag(const In* p, int lane) {
  return eight(p + 8 * lane);
}

// -------------------------------------------- global to LDS, by registers --
// A wave-uniform address as a scalar base formed here: with a 32-bit offset of
// the lane beside it, instead of a 64-bit pointer per lane carried over a loop.
// (The address space is named again: behind the asm the compiler would take
// the pointer for a generic one, and flat accesses wait on LDS too.)
typedef char __attribute__((address_space(1)))* gbytes;
__device__ __forceinline__ gbytes scalar_base(const void* p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  uint64_t v = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32 |
               (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u);
  asm volatile("" : "+s"(v));
  return reinterpret_cast<gbytes>(v);
}
typedef unsigned int gu32x2 __attribute__((ext_vector_type(2)));
typedef float gf32x4 __attribute__((ext_vector_type(4)));

// A part of a tensor as a buffer of `bytes` from p on: loads past its end
// return 0 and stores are dropped, so that tiles need no branches at the ends
// of a sequence (branches around loads make the compiler wait for them in
// turn).  Offsets are unsigned 32-bit bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint64_t v = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(v), 0, __builtin_amdgcn_readfirstlane(bytes),
                                           0x00027000);
}
constexpr uint32_t kNowhere = 0xfffffff0u;  // an offset past every buffer

// Eight floats, four and four of which 64 lanes lie side by side.
__device__ __forceinline__ void load_halves(gbytes p, Frag<float>& o) {
  const auto* q = reinterpret_cast<const gf32x4 __attribute__((address_space(1)))*>(p);
  const gf32x4 x = q[0], y = q[64];
#pragma unroll
  for (int j = 0; j < 4; ++j) { o.v[j] = x[j]; o.v[4 + j] = y[j]; }
}

// Four values in the input type, kept as such.
template <typename In>
struct Four;
template <>
struct Four<uint16_t> {
  uint32_t w[2];
  __device__ __forceinline__ void set(const float (&f)[4]) { w[0] = bf_pack(f[0], f[1]); w[1] = bf_pack(f[2], f[3]); }
  // as set, and f becomes what is left
  __device__ __forceinline__ void split(float (&f)[4]) { w[0] = split2(f[0], f[1]); w[1] = split2(f[2], f[3]); }
  __device__ __forceinline__ uint16_t get(int r) const { return (uint16_t)(w[r >> 1] >> (16 * (r & 1))); }
  __device__ __forceinline__ void put(uint16_t* p) const { *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]); }
  __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off) const {
    __builtin_amdgcn_raw_buffer_store_b64(gu32x2{w[0], w[1]}, r, off, 0, 0);
  }
};
template <>
struct Four<float> {
  float w[4];
  __device__ __forceinline__ void set(const float (&f)[4]) {
#pragma unroll
    for (int r = 0; r < 4; ++r) w[r] = f[r];
  }
  __device__ __forceinline__ float get(int r) const { return w[r]; }
  __device__ __forceinline__ void put(float* p) const { store_vec<float, 4>(p, w); }
  __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, uint32_t off) const {
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(gu32x4, gf32x4{w[0], w[1], w[2], w[3]}), r, off, 0, 0);
  }
};

// Eight consecutive columns of one row.
template <typename In>
struct Piece;
template <>
struct Piece<uint16_t> {
  uint4 v;
  // the first n values stay, the others become 0
  __device__ __forceinline__ void keep(int n) {
    auto part = [&](uint32_t w, int i) { return w & (n >= 2 * i + 2 ? ~0u : n == 2 * i + 1 ? 0xffffu : 0u); };
    v = make_uint4(part(v.x, 0), part(v.y, 1), part(v.z, 2), part(v.w, 3));
  }
  __device__ __forceinline__ void load_at(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    const auto w = __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
    v = make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ __forceinline__ void set(const uint16_t (&e)[8]) {
    v = make_uint4(e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16), e[4] | ((uint32_t)e[5] << 16),
                   e[6] | ((uint32_t)e[7] << 16));
  }
  __device__ __forceinline__ void get(uint16_t (&e)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { e[2 * j] = (uint16_t)w[j]; e[2 * j + 1] = (uint16_t)(w[j] >> 16); }
  }
  // columns 8 i .. 8 i + 7 of a tile row
  template <int COLS>
  __device__ __forceinline__ void put(const RowTile<uint16_t, COLS>& d, int row, int i) const {
    *reinterpret_cast<uint2*>(d.t + d.at(row, 2 * i)) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(d.t + d.at(row, 2 * i + 1)) = make_uint2(v.z, v.w);
  }
  template <int COLS>
  __device__ __forceinline__ void put(const ColTile<uint16_t, COLS>& d, int row, int i) const {
    *reinterpret_cast<uint4*>(d.t + d.at(row, 2 * i)) = v;
  }
  // an exponent of all ones somewhere: adding 1 to it carries into the sign
  __device__ __forceinline__ bool nonfinite() const {
    const uint32_t m = 0x7f807f80u, one = 0x00800080u;
    return ((((v.x & m) + one) | ((v.y & m) + one) | ((v.z & m) + one) | ((v.w & m) + one)) & 0x80008000u) != 0;
  }
  static __device__ __forceinline__ bool bad(uint16_t e) { return (e & 0x7f80u) == 0x7f80u; }
};
template <>
struct Piece<float> {
  float4 a, b;
  __device__ __forceinline__ void keep(int n) {
    a = make_float4(n > 0 ? a.x : 0.0f, n > 1 ? a.y : 0.0f, n > 2 ? a.z : 0.0f, n > 3 ? a.w : 0.0f);
    b = make_float4(n > 4 ? b.x : 0.0f, n > 5 ? b.y : 0.0f, n > 6 ? b.z : 0.0f, n > 7 ? b.w : 0.0f);
  }
  __device__ __forceinline__ void load_at(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    const gf32x4 x = __builtin_bit_cast(gf32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0));
    const gf32x4 y = __builtin_bit_cast(gf32x4, __builtin_amdgcn_raw_buffer_load_b128(r, off + 16, 0, 0));
    a = make_float4(x.x, x.y, x.z, x.w);
    b = make_float4(y.x, y.y, y.z, y.w);
  }
  __device__ __forceinline__ void set(const float (&e)[8]) {
    a = make_float4(e[0], e[1], e[2], e[3]);
    b = make_float4(e[4], e[5], e[6], e[7]);
  }
  __device__ __forceinline__ void get(float (&e)[8]) const {
    e[0] = a.x; e[1] = a.y; e[2] = a.z; e[3] = a.w; e[4] = b.x; e[5] = b.y; e[6] = b.z; e[7] = b.w;
  }
  template <typename Tile>
  __device__ __forceinline__ void put(const Tile& d, int row, int i) const {
    *reinterpret_cast<float4*>(d.t + d.at(row, 2 * i)) = a;
    *reinterpret_cast<float4*>(d.t + d.at(row, 2 * i + 1)) = b;
  }
  static __device__ __forceinline__ bool bad(float e) { return (__float_as_uint(e) & 0x7f800000u) == 0x7f800000u; }
  __device__ __forceinline__ bool nonfinite() const {
    return bad(a.x) || bad(a.y) || bad(a.z) || bad(a.w) || bad(b.x) || bad(b.y) || bad(b.z) || bad(b.w);
  }
};

// A ROWS x COLS tile through the registers of THREADS threads: load() issues
// the global loads, mask() zeroes what lies past the sequence or the width,
// store() writes the LDS tile.  VEC: 16-byte buffer loads (rows 16-byte
// aligned, width a multiple of 8, offsets in 32 bits); rows past the sequence
// read 0.
template <typename In, int ROWS, int COLS, int THREADS, bool VEC>
struct TileRegs {
  static constexpr int kPer = COLS / 8;                       // pieces of a row
  static constexpr int kN = (ROWS * kPer + THREADS - 1) / THREADS;
  Piece<In> r[kN];
  static_assert(THREADS % kPer == 0, "a thread keeps its columns");
  // Rows of 16 pieces are taken as two halves, so that 16 lanes write halves of
  // two rows (a RowTile's 8-byte writes then meet no bank twice).
  static __device__ __forceinline__ int row_of(int k, int tid = threadIdx.x) {
    const int r = kPer == 16 ? (tid >> 5) * 2 + ((tid >> 3) & 1) : tid / kPer;
    return r + k * (THREADS / kPer);
  }
  static __device__ __forceinline__ int col_of(int tid = threadIdx.x) {
    return (kPer == 16 ? (tid & 7) + ((tid >> 4) & 1) * 8 : tid % kPer) * 8;
  }
  // The thread's index as a value formed here: what is rarely needed is then
  // not kept in registers over a loop.
  static __device__ __forceinline__ int fresh_tid() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
  }
  // base: row 0, column 0 of the tile; `rows` of it are in the sequence (0:
  // nothing is loaded) and `cols` >= 1 columns are in the width
  __device__ __forceinline__ void load(const In* base, int64_t stride, int rows, int cols) {
    if constexpr (VEC) {
      const uint32_t st = (uint32_t)stride * (uint32_t)sizeof(In);
      const uint32_t off = (uint32_t)row_of(0) * st + (uint32_t)col_of() * (uint32_t)sizeof(In);
      const __amdgpu_buffer_rsrc_t buf =
          buffer_of(base, rows > 0 ? (uint32_t)(rows - 1) * st + (uint32_t)cols * (uint32_t)sizeof(In) : 0u);
#pragma unroll
      for (int k = 0; k < kN; ++k) r[k].load_at(buf, off + (uint32_t)(k * (THREADS / kPer)) * st);
    } else {
      if (rows == 0) return;
      const int tid = fresh_tid();
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int row = row_of(k, tid), col = col_of(tid);
        const In* p = base + (int64_t)(row < rows ? row : rows - 1) * stride;
        In e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = p[col + j < cols ? col + j : cols - 1];
        r[k].set(e);
      }
    }
  }
  __device__ __forceinline__ void mask(int rows, int cols) {
    if ((VEC || rows >= ROWS) && cols >= COLS) return;
    const int tid = fresh_tid();
#pragma unroll
    for (int k = 0; k < kN; ++k) r[k].keep(row_of(k, tid) < rows ? cols - col_of(tid) : 0);
  }
  template <typename Tile>
  __device__ __forceinline__ void store(const Tile& tile) const {
#pragma unroll
    for (int k = 0; k < kN; ++k)
      if (ROWS * kPer % THREADS == 0 || row_of(k) < ROWS) r[k].put(tile, row_of(k), col_of() / 8);
  }
  // Values that are not finite become 0; first[column] receives the first
  // row that held one.
  __device__ __forceinline__ void clean(int* first) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      if (r[k].nonfinite()) {
        const int tid = fresh_tid();
        In e[8];
        r[k].get(e);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (Piece<In>::bad(e[j])) {
            e[j] = In(0);
            atomicMin(first + col_of(tid) + j, row_of(k, tid));
          }
        r[k].set(e);
      }
    }
  }
};

// ------------------------------------------------------------ the chunk --
// Index of the wave in its workgroup, in a scalar register.
__device__ __forceinline__ int wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x >> 6); }

// Inclusive sum over the 64 lanes of a wave.
__device__ __forceinline__ float wave_scan(float v) {
  v += dpp_f<0x111>(v);  // row_shr:1, 2, 4, 8
  v += dpp_f<0x112>(v);
  v += dpp_f<0x114>(v);
  v += dpp_f<0x118>(v);
  // the last lane of rows 0 and 2 to rows 1 and 3, then of row 1 to rows 2, 3
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x142, 0xa, 0xf, false));
  v += __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x143, 0xc, 0xf, false));
  return v;
}
__device__ __forceinline__ float last_lane(float v) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

// Sums over the lanes of a 16-lane row: this lane and those after it; those
// before it (from their own terms alone: neither is the difference of two sums).
__device__ __forceinline__ float row_from(float v) {
  v += dpp_f<0x101>(v);  // row_shl:1, 2, 4, 8
  v += dpp_f<0x102>(v);
  v += dpp_f<0x104>(v);
  v += dpp_f<0x108>(v);
  return v;
}
__device__ __forceinline__ float row_before(float v) {
  v += dpp_f<0x111>(v);  // row_shr:1, 2, 4, 8
  v += dpp_f<0x112>(v);
  v += dpp_f<0x114>(v);
  v += dpp_f<0x118>(v);
  return dpp_f<0x111>(v);
}
// Rows 4 g .. 4 g + 3 of column c, as a lane holds them of a 16 x 16 tile: for
// each row t the column's sum over row t and those after it, 0 unless c < t.
// Added over a row's lanes this is the tile's part with rows from t on and
// columns before t.
__device__ __forceinline__ void corner(float (&v)[4], int g, int c) {
  float run = 0.0f;
#pragma unroll
  for (int r = 3; r >= 0; --r) {
    run += c < 4 * g + r ? v[r] : 0.0f;
    v[r] = run;
  }
  // the later row groups: the other of the pair, then the upper pair
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(run), __float_as_uint(run), false, false);
  const float both = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(both), __float_as_uint(both), false, false);
  const float later = ((g & 1) ? 0.0f : __uint_as_float(p[1])) + (g < 2 ? __uint_as_float(q[1]) : 0.0f);
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = c < 4 * g + r ? v[r] + later : 0.0f;
}

// A running sum of log2 decays in two floats.  `hi` sums multiples of 2^-9,
// exactly up to 2^15 (128 tokens of at most 150), `lo` the rests of at most
// 2^-10 each.  So the difference of two sums is good to 2^-24 of itself, however
// much the chunk decays beside it: one float would leave 2^-24 of the chunk's
// whole sum in every decay, 7e-5 of it behind eight resets.
struct LogSum {
  float hi, lo;
};
__device__ __forceinline__ LogSum log_scan(float v) {
  const float hi = rintf(v * 512.0f) * (1.0f / 512.0f);
  return {wave_scan(hi), wave_scan(v - hi)};
}
__device__ __forceinline__ LogSum last_lane(LogSum v) { return {last_lane(v.hi), last_lane(v.lo)}; }
// The decay from sum b on to sum a.
__device__ __forceinline__ float decay_between(float a_hi, float a_lo, float b_hi, float b_lo) {
  return fast_exp2((a_hi - b_hi) + (a_lo - b_lo));
}
__device__ __forceinline__ float decay_between(LogSum a, LogSum b) { return decay_between(a.hi, a.lo, b.hi, b.lo); }

struct HeadsArgs {
  const void* x;
  const void* delta;      // or null (step 1)
  const float* dbias;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* D;         // or null
  const float* h0;        // (batch, heads, headdim, dstate) or null
  const float* dh_last;   // the same, backward
  const void* dy;         // contiguous, backward
  void* y;
  float* h_last;          // or null
  float* dh0;             // or null, backward
  int softplus, unit;
  int heads, headdim, ptiles, hpg, dstate;  // ptiles: 64-channel tiles of a head; hpg: heads per group
  int64_t batch, L;
  int64_t rows, row0;     // rows of the call, first row of this launch
  int64_t x_batch, x_token, d_batch, d_token, b_batch, b_token, c_batch, c_token;
  int64_t nseg, seg_len;  // segments along L (a multiple of the stored blocks)
  float* agg;             // segment states from zero (dir, seg, row, 64, NT)
  float* sd;              // and their summed log2 decays (dir, seg, row)
  float* hin;             // state entering each segment (dir, seg, row, 64, NT) or null
  float* planes;          // stored states of the backward, see heads_bwd.hip
};

// A row of the launch: one 64-channel tile of one head of one sequence.
struct HeadRow {
  int64_t row, b;
  int hd, pt, grp;
};
__device__ __forceinline__ HeadRow head_row(const HeadsArgs& a, int64_t row) {
  HeadRow o;
  o.row = row;
  const int64_t bh = row / a.ptiles;
  o.pt = (int)(row - bh * a.ptiles);
  o.b = bh / a.heads;
  o.hd = (int)(bh - o.b * a.heads);
  o.grp = o.hd / a.hpg;
  return o;
}

// The stored step of token `lane` of `rows`, at p with stride `st` (elements).
template <typename In, bool VEC>
__device__ __forceinline__ void load_step(In& raw, const In* p, int64_t st, int lane, int rows) {
  if constexpr (VEC) {
    const __amdgpu_buffer_rsrc_t buf =
        buffer_of(p, rows > 0 ? ((uint32_t)(rows - 1) * (uint32_t)st + 1) * (uint32_t)sizeof(In) : 0u);
    const uint32_t off = (uint32_t)lane * (uint32_t)st * (uint32_t)sizeof(In);
    if constexpr (sizeof(In) == 2)
      raw = __builtin_amdgcn_raw_buffer_load_b16(buf, off, 0, 0);
    else
      raw = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(buf, off, 0, 0));
  } else {
    if (lane < rows) raw = p[lane * st];
  }
}

// Step of a token of head hd: raw is the stored delta (or unused).
__device__ __forceinline__ float step_of(const HeadsArgs& a, float raw, float bias) {
  if (!a.delta) return 1.0f;
  const float v = raw + bias;
  return a.softplus ? softplus_f(v) : v;
}

// ------------------------------------------------------------ host side --
struct HeadsPlan {
  int NT;             // padded state width: 32, 64 or 128
  int64_t rows;       // batch * heads * ptiles
  int64_t ptiles;
  bool vec;
};
HeadsPlan heads_plan(const s6_heads_dims& d, int in_dtype, const void* x, const void* Bm, const void* Cm, const void* dy);
HeadsArgs heads_args(const s6_heads_dims& d, const HeadsPlan& p, int flags, const void* x, const void* delta,
                     const float* dbias, const float* A, const void* Bm, const void* Cm, const float* D,
                     const float* h0);

// Launches of at most this many workgroups: a launch counts its work items in 32
// bits, and one of more wraps without an error.
constexpr int64_t kMaxBlocks = int64_t(1) << 22;

// Segments along L for `rows` rows, each a multiple of `unit` tokens.
void heads_segments(int64_t rows, int64_t L, int64_t unit, int64_t* nseg, int64_t* seg_len);

// The state walk over every segment in one or both directions, see
// heads_state.hip.  mode 0: end states from zero (agg, sd); mode 1: from hin
// (or h0 / dh_last), storing the planes; dirs: 1 (forward in time) or 2.
int launch_heads_state(int in_dtype, const HeadsArgs& a, const HeadsPlan& p, int mode, int dirs, hipStream_t st);
// hin of every segment from h0 (or dh_last, direction 1), agg and sd.
int launch_heads_fold(const HeadsArgs& a, const HeadsPlan& p, int dirs, hipStream_t st);

}  // namespace s6i

#endif  // S6_HEADS_KERNEL_H_
