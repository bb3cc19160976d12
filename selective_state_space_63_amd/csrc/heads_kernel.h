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
// operand of the next product in registers, without a shuffle.  LDS tiles
// keep their columns in that order (chunks of four: 0, 4, 1, 5, 2, 6, 3, 7 of
// each 32), so an operand along a row is one 16-byte read per lane; an operand
// down a column is read with the transposing LDS read.
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
constexpr int kPad = 8;      // LDS row padding in elements (rows an odd number of 16-byte units apart)

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
__device__ __forceinline__ void to_pair(const float (&f)[8], Pair<uint16_t>& o) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const __bf16 h = (__bf16)f[j];
    o.hi.v[j] = h;
    o.lo.v[j] = (__bf16)(f[j] - (float)h);
  }
}
__device__ __forceinline__ void to_pair(const float (&f)[8], Pair<float>& o) { to_frag(f, o.hi); }

// d += (hi + lo) b  and  d += a (hi + lo)
__device__ __forceinline__ f32x4 mma_pair(const Pair<uint16_t>& a, const Frag<uint16_t>& b, f32x4 d) {
  return mma(a.lo, b, mma(a.hi, b, d));
}
__device__ __forceinline__ f32x4 mma_pair(const Frag<uint16_t>& a, const Pair<uint16_t>& b, f32x4 d) {
  return mma(a, b.lo, mma(a, b.hi, d));
}
__device__ __forceinline__ f32x4 mma_pair(const Pair<float>& a, const Frag<float>& b, f32x4 d) { return mma(a.hi, b, d); }
__device__ __forceinline__ f32x4 mma_pair(const Frag<float>& a, const Pair<float>& b, f32x4 d) { return mma(a, b.hi, d); }

// ------------------------------------------------------------- LDS tiles --
// Offset of the four-column chunk m (columns 4 m .. 4 m + 3) in a tile row.
__device__ __forceinline__ int chunk_at(int m) { return (m & ~7) * 4 + ((m & 3) * 2 + ((m >> 2) & 1)) * 4; }

// K = columns 32 kk .. 32 kk + 31 of row `row`.
__device__ __forceinline__ Frag<uint16_t> row_frag(const uint16_t* t, int pitch, int row, int kk, int g) {
  Frag<uint16_t> o;
  o.v = *reinterpret_cast<const bf16x8*>(t + row * pitch + 32 * kk + 8 * g);
  return o;
}
__device__ __forceinline__ Frag<float> row_frag(const float* t, int pitch, int row, int kk, int g) {
  Frag<float> o;
  const float4* p = reinterpret_cast<const float4*>(t + row * pitch + 32 * kk + 8 * g);
  const float4 x = p[0], y = p[1];
  o.v[0] = x.x; o.v[1] = x.y; o.v[2] = x.z; o.v[3] = x.w;
  o.v[4] = y.x; o.v[5] = y.y; o.v[6] = y.z; o.v[7] = y.w;
  return o;
}

// K = rows 32 kk .. 32 kk + 31 of column 16 q + c.  bf16: the transposing
// read gives each lane four rows of its column, from 8-byte pieces that the
// 16 lanes of a group fetch (lane i: row i / 4 of the four, chunk i % 4 of the
// sixteen columns).
__device__ __forceinline__ Frag<uint16_t> col_frag(const uint16_t* t, int pitch, int q, int kk, int g, int c) {
  const uint16_t* p = t + (32 * kk + 4 * g + (c >> 2)) * pitch + chunk_at(4 * q + (c & 3));
  typedef __attribute__((address_space(3))) s16x4* lds4;
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uint16_t*)p);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4)(uint16_t*)(p + 16 * pitch));
  Frag<uint16_t> o;
  o.v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
  return o;
}
__device__ __forceinline__ Frag<float> col_frag(const float* t, int pitch, int q, int kk, int g, int c) {
  const float* p = t + (32 * kk + 4 * g) * pitch + chunk_at(4 * q + (c >> 2)) + (c & 3);
  Frag<float> o;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    o.v[j] = p[j * pitch];
    o.v[4 + j] = p[(16 + j) * pitch];
  }
  return o;
}

// Four columns 4 m .. 4 m + 3 of a row as floats.
template <typename In>
__device__ __forceinline__ void row_four(const In* t, int pitch, int row, int m, float (&f)[4]) {
  load_vec<In, 4>(t + row * pitch + chunk_at(m), f);
}

// An operand kept in LDS as such: 8 values per lane.
__device__ __forceinline__ Frag<uint16_t> lane_frag(const uint16_t* p, int lane) {
  Frag<uint16_t> o;
  o.v = *reinterpret_cast<const bf16x8*>(p + 8 * lane);
  return o;
}
__device__ __forceinline__ Frag<float> lane_frag(const float* p, int lane) {
  return row_frag(p + 8 * lane, 0, 0, 0, 0);
}

// -------------------------------------------- global to LDS, by registers --
// Eight consecutive columns of one row.
template <typename In>
struct Piece;
template <>
struct Piece<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void set(const uint16_t (&e)[8]) {
    v = make_uint4(e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16), e[4] | ((uint32_t)e[5] << 16),
                   e[6] | ((uint32_t)e[7] << 16));
  }
  __device__ __forceinline__ void get(uint16_t (&e)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) { e[2 * j] = (uint16_t)w[j]; e[2 * j + 1] = (uint16_t)(w[j] >> 16); }
  }
  __device__ __forceinline__ void store(uint16_t* row, int i) const {
    *reinterpret_cast<uint2*>(row + chunk_at(2 * i)) = make_uint2(v.x, v.y);
    *reinterpret_cast<uint2*>(row + chunk_at(2 * i + 1)) = make_uint2(v.z, v.w);
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
  __device__ __forceinline__ void zero() { a = b = make_float4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void set(const float (&e)[8]) {
    a = make_float4(e[0], e[1], e[2], e[3]);
    b = make_float4(e[4], e[5], e[6], e[7]);
  }
  __device__ __forceinline__ void get(float (&e)[8]) const {
    e[0] = a.x; e[1] = a.y; e[2] = a.z; e[3] = a.w; e[4] = b.x; e[5] = b.y; e[6] = b.z; e[7] = b.w;
  }
  __device__ __forceinline__ void store(float* row, int i) const {
    *reinterpret_cast<float4*>(row + chunk_at(2 * i)) = a;
    *reinterpret_cast<float4*>(row + chunk_at(2 * i + 1)) = b;
  }
  static __device__ __forceinline__ bool bad(float e) { return (__float_as_uint(e) & 0x7f800000u) == 0x7f800000u; }
  __device__ __forceinline__ bool nonfinite() const {
    return bad(a.x) || bad(a.y) || bad(a.z) || bad(a.w) || bad(b.x) || bad(b.y) || bad(b.z) || bad(b.w);
  }
};

// A ROWS x COLS tile through the registers of THREADS threads: load() issues
// the global loads (rows past the sequence and columns past the width are
// zero), store() writes the LDS tile.  VEC: 16-byte loads (rows 16-byte
// aligned, width a multiple of 8).
template <typename In, int ROWS, int COLS, int THREADS, bool VEC>
struct TileRegs {
  static constexpr int kPer = COLS / 8;                       // pieces of a row
  static constexpr int kN = (ROWS * kPer + THREADS - 1) / THREADS;
  Piece<In> r[kN];
  // base: row 0, column 0 of the tile; `rows` of it are in the sequence and
  // `cols` columns are in the width
  __device__ __forceinline__ void load(const In* base, int64_t stride, int rows, int cols) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int id = k * THREADS + threadIdx.x;
      const int row = id / kPer, col = (id % kPer) * 8;
      r[k].zero();
      if (row < rows && row < ROWS) {
        const In* p = base + (int64_t)row * stride + col;
        if constexpr (VEC) {
          if (col < cols) r[k].load(p);
        } else {
          In e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) e[j] = col + j < cols ? p[j] : In(0);
          r[k].set(e);
        }
      }
    }
  }
  __device__ __forceinline__ void store(In* tile, int pitch) const {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      const int id = k * THREADS + threadIdx.x;
      const int row = id / kPer;
      if (ROWS * kPer % THREADS == 0 || row < ROWS) r[k].store(tile + row * pitch, id % kPer);
    }
  }
  // Values that are not finite become 0; first[column] receives the first
  // row that held one, *any is set.  Returns whether there was one.
  __device__ __forceinline__ void clean(int* first, int* any) {
#pragma unroll
    for (int k = 0; k < kN; ++k) {
      if (r[k].nonfinite()) {
        const int id = k * THREADS + threadIdx.x;
        In e[8];
        r[k].get(e);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (Piece<In>::bad(e[j])) {
            e[j] = In(0);
            atomicMin(first + (id % kPer) * 8 + j, id / kPer);
          }
        r[k].set(e);
        *any = 1;
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
  int64_t x_batch, x_token, d_batch, d_token, b_batch, b_token, c_batch, c_token;
  int64_t nseg, seg_len;  // segments along L (a multiple of the stored blocks)
  float* agg;             // segment states from zero (dir, seg, row, 64, NT)
  float* sd;              // and their summed log2 decays (dir, seg, row)
  float* hin;             // state entering each segment (dir, seg, row, 64, NT) or null
  void* planes;           // stored states of the backward, see heads_bwd.hip
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
