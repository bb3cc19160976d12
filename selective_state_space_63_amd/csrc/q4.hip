// q4.hip -- products of few rows with 4-bit weights and group scales, and
// their packing (include/s6_q4.h).
//
//   y[t, n] = sum over groups G of scale[n, G] * sum_{k in G} x[t, k] value[n, k]
//
// Bound by the weights' bytes at few rows, so the weights go from memory to
// registers once, as codes, 16 bytes per lane; the conversion instruction
// turns two codes into two bf16 (exact), and the matrix cores multiply: 16
// weight rows by 16 rows of x, 32 columns an instruction.  A code's value is
// exact in bf16, so are its products with bf16 (fp32 sums); the scales, which
// are not, multiply the sums of their groups in fp32.
//
// A group's sum may be 128 * 6 times the largest x before its scale makes it
// small: values are converted as 2^-10 of themselves where x is fp32 or bf16,
// whose largest is fp32's, and the result is multiplied by 2^10.  Both are exact:
// bf16 are multiples of 2^-133, so the products are of 2^-144; a result below 2^-116
// rounds to 2^-139.
#include "s6_q4.h"

#include "block_internal.h"

namespace s6i {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

struct Q4Args {
  const void* x;
  const float* x_scale;
  const uint8_t* codes;
  const uint16_t* scales;
  void* y;
  int64_t rows, outer, x_stride;
  int inner;
  int fine;       // log2(128 / group)
  int ngroups;    // inner / group
  int64_t base;   // first tile of weight rows of the launch
  int wide;       // rows of y begin at 16 bytes
  int slice;      // blocks of columns of a slice
  float* parts;   // the slices' sums (slices, rows, outer), or null
  float up;       // what sums are multiplied by without x_scale: 1 / kDown of x's type
};

// What values are multiplied by when they are converted.
template <typename XT>
constexpr float kDown = sizeof(XT) == 1 ? 1.0f : 0x1p-10f;

// Eight codes as bf16.
template <typename XT>
__device__ __forceinline__ bf16x8 values8(uint32_t c) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, kDown<XT>, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, kDown<XT>, 1);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, kDown<XT>, 2);
  const bf16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, kDown<XT>, 3);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}
// Eight e4m3 values as bf16.
__device__ __forceinline__ bf16x8 bytes8(uint32_t lo, uint32_t hi) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));

// A part of a tensor as a buffer of `bytes` from p on: loads past its end
// return 0.  Offsets are unsigned 32-bit bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_at(const void* p, uint32_t bytes) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint64_t v = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32 |
                     (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u);
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(v), 0, __builtin_amdgcn_readfirstlane(bytes),
                                           0x00027000);
}
// Offsets past every buffer (each is below 2^28 bytes): of a row that does not
// exist, and of columns; their sum is one too.
constexpr uint32_t kNoRow = 0x80000000u, kNoColumn = 0x40000000u;
constexpr int64_t kMaxStride = 1 << 20;   // most columns, and elements from row to row
template <typename XT>
constexpr bool rows_fit(int rows) { return rows * kMaxStride * (int64_t)sizeof(XT) < 1 << 28; }
static_assert(16 * (kMaxStride / 2) < 1 << 28 && 16 * (kMaxStride / 32) * 2 < 1 << 28, "16 weight rows, and their scales");
constexpr int kFewRows = 16;              // most rows of the few-row kernel

// Eight consecutive values of x as loaded, and as bf16 parts whose sum they are.
template <typename XT, bool XV>
struct X8 {
  static constexpr int kParts = sizeof(XT) == 4 ? 3 : 1;
  alignas(16) XT e[8];
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (XV && sizeof(XT) == 1) {
      const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
      __builtin_memcpy(e, &v, 8);
    } else if constexpr (XV) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(XT) / 2; ++i) {
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(r, off + 16 * i, 0, 0);
        __builtin_memcpy(reinterpret_cast<char*>(e) + 16 * i, &v, 16);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if constexpr (sizeof(XT) == 4) e[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off + 4 * i, 0, 0));
        else if constexpr (sizeof(XT) == 2) e[i] = __builtin_amdgcn_raw_buffer_load_b16(r, off + 2 * i, 0, 0);
        else e[i] = __builtin_amdgcn_raw_buffer_load_b8(r, off + i, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void get(bf16x8 (&o)[kParts]) const {
    if constexpr (sizeof(XT) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // the first part is cut, which rounds nothing up to infinity, and what a
        // part leaves is exact; a value that is not finite stays in the first
        const float cut = __uint_as_float(__float_as_uint(e[i]) & 0xffff0000u);
        const float left = e[i] - cut;
        const bool fin = __builtin_fabsf(left) < __builtin_inff();
        const float r = fin ? left : 0.0f;
        const __bf16 h = (__bf16)(fin ? cut : e[i]);
        const __bf16 m = (__bf16)r;
        o[0][i] = h;
        o[1][i] = m;
        o[2][i] = (__bf16)(r - (float)m);
      }
    } else if constexpr (sizeof(XT) == 2) {
      __builtin_memcpy(&o[0], e, 16);
    } else {
      uint2 v;
      __builtin_memcpy(&v, e, 8);
      o[0] = bytes8(v.x, v.y);
    }
  }
};

// Words (q, j) <-> (j, q) between the wave's four rows of 16 lanes and four
// registers.
__device__ __forceinline__ void transpose4(uint32_t (&c)[4]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const auto r = __builtin_amdgcn_permlane32_swap(c[i], c[i + 2], false, false);
    c[i] = r[0]; c[i + 2] = r[1];
  }
#pragma unroll
  for (int i = 0; i < 4; i += 2) {
    const auto r = __builtin_amdgcn_permlane16_swap(c[i], c[i + 1], false, false);
    c[i] = r[0]; c[i + 1] = r[1];
  }
}

constexpr int kBlk = 128;  // columns of a block: 16 bytes of codes per lane, four matrix instructions

// 16 weight rows from n0 on.  Lane l has row l % 16 and, of a block of
// columns, 32 codes from 32 (l / 16) on.  FINE (groups of 32 or 64): the codes are
// transposed so that step j's 32 columns, 32 j to + 31, lie in one group; else
// step j takes columns 8 j to + 7 of each lane's 32, all in the block's group.
template <bool FINE>
struct WRows {
  __amdgpu_buffer_rsrc_t codes, scales;
  uint32_t code_at, scale_at;
  int q32, fine;  // q32: first of the lane's columns in a block; fine: log2 of 128 / group
  __device__ __forceinline__ WRows(const Q4Args& a, int64_t n0) {
    const int lane = threadIdx.x & 63, i = lane & 15;
    q32 = 2 * (lane & 48);
    const int64_t left = a.outer - n0;
    const uint32_t rows = left < 0 ? 0 : left < 16 ? (uint32_t)left : 16;
    const uint32_t row = (uint32_t)a.inner >> 1;
    codes = buffer_at(a.codes + n0 * row, rows * row);
    scales = buffer_at(a.scales + n0 * a.ngroups, rows * (uint32_t)a.ngroups * 2);
    code_at = i * row + (q32 >> 1);
    scale_at = i * (uint32_t)a.ngroups * 2;
    fine = a.fine;
  }
  struct Block {
    uint32_t c[4];
    uint32_t s;  // scale: of the block's group, or (FINE) of the group of the lane's 32 columns
  };
  // Block b; what lies past column `end` is 0.
  __device__ __forceinline__ void load(Block& o, int b, int end) const {
    const int k = b * kBlk;
    uint32_t at = code_at + (k < end ? (uint32_t)k >> 1 : kNoColumn), sat;
    if constexpr (FINE) {
      const bool on = k + q32 < end;
      at = on ? at : kNoColumn;
      sat = on ? scale_at + ((uint32_t)(k + q32) >> 7 - fine) * 2 : kNoColumn;
    } else {
      sat = scale_at + (k < end ? (uint32_t)b * 2 : kNoColumn);
    }
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(codes, at, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) o.c[j] = v[j];
    o.s = __builtin_amdgcn_raw_buffer_load_b16(scales, sat, 0, 0);
  }
};
// The scales of the four steps of a block (FINE), or of the block.
template <bool FINE>
__device__ __forceinline__ void scales_of(uint32_t s, float (&f)[4]) {
  if constexpr (FINE) {  // the four rows of 16 lanes to all of them
    const auto a = __builtin_amdgcn_permlane16_swap(s << 16, s << 16, false, false);
    const auto b = __builtin_amdgcn_permlane32_swap(a[0], a[0], false, false);
    const auto c = __builtin_amdgcn_permlane32_swap(a[1], a[1], false, false);
    f[0] = __uint_as_float(b[0]); f[1] = __uint_as_float(c[0]);
    f[2] = __uint_as_float(b[1]); f[3] = __uint_as_float(c[1]);
  } else {
    f[3] = __uint_as_float(s << 16);
  }
}

// Few rows, 16 at most.  A workgroup has 16 weight rows; its waves take the
// blocks of columns in turn, U of them loaded together, and their
// sums meet in LDS in a fixed order.  An instruction multiplies 16 rows of x
// (first operand) by 16 weight rows: lane l gets the sums of x rows 4 (l / 16)
// to + 3 and weight row l % 16, whose scale is then the lane's own.  Rows and
// columns that do not exist are loaded as 0 through the buffers' ends.
// One bf16 row of 2560 to 10576: 6.3 us (floor 2.2: 14 MB of codes), a launch and
// the latency of loads that are all under way at once; 16 rows 11.4, 16 of 5120 to
// 2560 in groups of 32 9.4 (1.2): x is read again for every 16 weight rows, 54 MB
// of it for 16 rows of 2560 to 10576.  One fp32 row 12.6: it is split again there too.
template <typename XT, bool FINE, bool XV, typename YT>
__global__ __launch_bounds__(1024) void s6_q4_few_kernel(Q4Args a) {
  extern __shared__ float part[];  // (W - 1, 64, 4)
  using X = X8<XT, XV>;
  constexpr int U = sizeof(XT) == 4 ? 2 : 4;
  constexpr uint32_t kE = sizeof(XT);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
  const int i = lane & 15, q = lane >> 4;
  const int64_t n0 = (a.base + blockIdx.x) * 16;
  const WRows<FINE> wr(a, n0);
  static_assert(rows_fit<XT>(kFewRows), "x's buffer");
  const int rows = (int)a.rows;
  const uint32_t step = (uint32_t)a.x_stride * kE;
  const __amdgpu_buffer_rsrc_t xb = buffer_at(a.x, (uint32_t)(rows - 1) * step + (uint32_t)a.inner * kE);
  const uint32_t x_at = i < rows ? i * step + (FINE ? 8 : 32) * q * kE : kNoRow;
  f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
  const int nb = (a.inner + kBlk - 1) / kBlk;
  for (int b0 = wave; b0 < nb; b0 += U * W) {
    typename WRows<FINE>::Block wb[U];
    X xr[U][4];
#pragma unroll
    for (int v = 0; v < U; ++v) wr.load(wb[v], b0 + v * W, a.inner);
#pragma unroll
    for (int v = 0; v < U; ++v)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = (b0 + v * W) * kBlk + (FINE ? 32 : 8) * j;
        xr[v][j].load(xb, x_at + (k < a.inner ? (uint32_t)k * kE : kNoColumn));
      }
#pragma unroll
    for (int v = 0; v < U; ++v) {
      if constexpr (FINE) transpose4(wb[v].c);
      float sc[4];
      scales_of<FINE>(wb[v].s, sc);
      f32x4 acc;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 w = values8<XT>(wb[v].c[j]);
        bf16x8 xp[X::kParts];
        xr[v][j].get(xp);
        if (FINE || j == 0) acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int p = X::kParts - 1; p >= 0; --p) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xp[p], w, acc, 0, 0, 0);
        if (FINE || j == 3) {
#pragma unroll
          for (int r = 0; r < 4; ++r) sum[r] = __builtin_fmaf(sc[j], acc[r], sum[r]);
        }
      }
    }
  }
  f32x4* parts = reinterpret_cast<f32x4*>(part);
  if (wave > 0) parts[(wave - 1) * 64 + lane] = sum;
  __syncthreads();
  if (wave > 0 || n0 + i >= a.outer) return;
#pragma unroll 4
  for (int w = 0; w + 1 < W; ++w) sum += parts[w * 64 + lane];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t t = 4 * q + r;
    if (t >= a.rows) continue;
    const float xs = a.x_scale ? a.x_scale[t] : a.up;
    static_cast<YT*>(a.y)[t * a.outer + n0 + i] = from_f32<YT>(sum[r] * xs);
  }
}

// More rows.  A workgroup has 128 weight rows and BM rows of x, and takes two
// blocks of columns a turn, four waves to each (32 weight rows to a wave): the
// blocks of x pass through LDS as bf16, a turn's loads under way during the turn
// before, and each piece that a wave reads meets both of its tiles of weight
// rows.  The two halves' sums meet in LDS, from where y is stored in whole
// lines.  blockIdx.z: a slice of the columns, its sums left in the workspace
// where there are several.
//
// 256 8-bit rows of 2560 to 10576, groups of 128: 27 us (floor 10), of which 3 the launch,
// 5 before and after the turns.  LDS reads, conversions and products would take
// 7.4, 6.5 and 5.5 us of each CU; with two waves per SIMD that meet at every
// turn they mostly go one after another.  One block a turn without halves: 34 us;
// x straight to registers, every wave all of a tile's rows: 42 us (16 bytes of
// each of 16 rows a load); more blocks under way from memory: no change.
constexpr int kBN = 128;
// Pitch of a row of x in LDS: 16 bytes of each of 16 rows lie in all banks once.
// Some accesses meet all the same, as lanes are not served in the order of rows:
// SQ_LDS_BANK_CONFLICT is 14 % of the busy cycles (256 8-bit rows of 2560 to 10576).
constexpr int kXP = kBlk + 8;
constexpr int kYP = kBN + 4;   // pitch of a row of sums
constexpr size_t many_lds(int bm, int parts) { return (size_t)2 * 2 * parts * bm * kXP * sizeof(uint16_t); }
static_assert(many_lds(32, 1) >= 32 * kYP * sizeof(float), "the sums take the place of x");
// Waves per SIMD, which the registers leave room for (smaller groups of bf16 rows
// spill at four: 136 rows of 2560 to 10576, groups of 32, 27.5 us, else 22.2).
template <typename XT, int BM, bool FINE>
constexpr int kManyWaves = BM > 64 || (BM == 64 && FINE && sizeof(XT) == 2) ? 2 : 4;
template <typename XT, int BM, bool FINE, bool XV, typename YT>
__global__ __launch_bounds__(512, (kManyWaves<XT, BM, FINE>)) void s6_q4_many_kernel(Q4Args a) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  using X = X8<XT, XV>;
  using Tile = uint16_t(*)[kXP];
  constexpr uint32_t kE = sizeof(XT);
  constexpr int M = BM / 16, NP = X::kParts;
  static_assert(rows_fit<XT>(BM), "x's buffer");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), half = wave >> 2;
  const int i = lane & 15, q = lane >> 4;
  const int64_t m0 = (a.base + blockIdx.x) * kBN, t0 = (int64_t)blockIdx.y * BM;
  const int n0 = 32 * (wave & 3);
  const WRows<FINE> w0(a, m0 + n0), w1(a, m0 + n0 + 16);
  const int rows = a.rows - t0 < BM ? (int)(a.rows - t0) : BM;
  const uint32_t step = (uint32_t)a.x_stride * kE;
  const __amdgpu_buffer_rsrc_t xb =
      buffer_at(static_cast<const XT*>(a.x) + t0 * a.x_stride, (uint32_t)(rows - 1) * step + (uint32_t)a.inner * kE);
  const int nb = (a.inner + kBlk - 1) / kBlk;
  const int lo = blockIdx.z * a.slice, hi = lo + a.slice < nb ? lo + a.slice : nb;
  // what lies past the slice is 0 (no branch around loads, which would make
  // them wait for one another)
  const int end = (int64_t)hi * kBlk < a.inner ? hi * kBlk : a.inner;
  // staging: a thread has eight columns, 8 (c % 16) on, of rows c / 16 + 16 m of
  // its half's block
  const int c = threadIdx.x & 255, sc = 8 * (c & 15), sr = c >> 4;
  X xr[M];
  typename WRows<FINE>::Block wb[2];
  uint32_t x_at[M];
#pragma unroll
  for (int m = 0; m < M; ++m) x_at[m] = sr + 16 * m < rows ? (sr + 16 * m) * step + sc * kE : kNoRow;
  auto load = [&](int b) {
    w0.load(wb[0], b, end);
    w1.load(wb[1], b, end);
    const int k = b * kBlk;
#pragma unroll
    for (int m = 0; m < M; ++m)
      xr[m].load(xb, FINE ? (k + sc < end ? x_at[m] + (uint32_t)k * kE : kNoColumn)
                          : x_at[m] + (k < end ? (uint32_t)k * kE : kNoColumn));
  };
  f32x4 sum[2][M];
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int u = 0; u < M; ++u) sum[h][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  load(lo + half);
  for (int b = lo; b < hi; b += 2) {
    Tile x = reinterpret_cast<Tile>(lds) + (((b - lo) & 2) + half) * (NP * BM);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      bf16x8 v[NP];
      xr[m].get(v);
#pragma unroll
      for (int p = 0; p < NP; ++p) *reinterpret_cast<bf16x8*>(&x[p * BM + sr + 16 * m][sc]) = v[p];
    }
    typename WRows<FINE>::Block c0 = wb[0], c1 = wb[1];
    // (a turn's tiles were last read two turns ago, before the barrier of the
    // turn between)
    __syncthreads();
    load(b + 2 + half);
    if constexpr (FINE) {
      transpose4(c0.c);
      transpose4(c1.c);
    }
    float s0[4], s1[4];
    scales_of<FINE>(c0.s, s0);
    scales_of<FINE>(c1.s, s1);
    f32x4 acc[2][M];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8 v0 = values8<XT>(c0.c[j]), v1 = values8<XT>(c1.c[j]);
#pragma unroll
      for (int u = 0; u < M; ++u) {
        if (FINE || j == 0) acc[0][u] = acc[1][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int p = NP - 1; p >= 0; --p) {
          const bf16x8 xv =
              *reinterpret_cast<const bf16x8*>(&x[p * BM + 16 * u + i][FINE ? 32 * j + 8 * q : 32 * q + 8 * j]);
          acc[0][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, v0, acc[0][u], 0, 0, 0);
          acc[1][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, v1, acc[1][u], 0, 0, 0);
        }
      }
      if (FINE || j == 3) {
#pragma unroll
        for (int u = 0; u < M; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sum[0][u][r] = __builtin_fmaf(s0[j], acc[0][u][r], sum[0][u][r]);
            sum[1][u][r] = __builtin_fmaf(s1[j], acc[1][u][r], sum[1][u][r]);
          }
      }
    }
  }
  float(*ys)[kYP] = reinterpret_cast<float(*)[kYP]>(lds);
  __syncthreads();
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    if (half == pass) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int u = 0; u < M; ++u)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            float* p = &ys[16 * u + 4 * q + r][n0 + 16 * h + i];
            *p = pass == 0 ? sum[h][u][r] : *p + sum[h][u][r];
          }
    }
    __syncthreads();
  }
  // eight columns of a row to a thread
  const int64_t left = a.outer - m0;
  const bool wide = a.wide && left >= kBN;
#pragma unroll
  for (int m = 0; m < BM / 32; ++m) {
    const int t = (threadIdx.x >> 4) + 32 * m, n = 8 * (threadIdx.x & 15);
    if (t >= rows) continue;
    float v[8];
    load_vec<float, 8>(&ys[t][n], v);
    const float xs = a.parts ? 1.0f : a.x_scale ? a.x_scale[t0 + t] : a.up;
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= xs;
    const int64_t at = (t0 + t) * a.outer + m0 + n;
    if (a.parts) {
      float* p = a.parts + (int64_t)blockIdx.z * a.rows * a.outer + at;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < left) p[e] = v[e];
    } else if (wide) {
      store_vec<YT, 8>(static_cast<YT*>(a.y) + at, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (n + e < left) static_cast<YT*>(a.y)[at + e] = from_f32<YT>(v[e]);
    }
  }
}

// y from the slices' sums, in a fixed order.
template <typename YT>
__global__ __launch_bounds__(256) void s6_q4_join_kernel(Q4Args a, int slices) {
  const int64_t n = (int64_t)blockIdx.x * 256 + threadIdx.x, t = blockIdx.y, all = a.rows * a.outer;
  if (n >= a.outer) return;
  float s = 0.0f;
#pragma unroll 4
  for (int z = 0; z < slices; ++z) s += a.parts[z * all + t * a.outer + n];
  static_cast<YT*>(a.y)[t * a.outer + n] = from_f32<YT>(s * (a.x_scale ? a.x_scale[t] : a.up));
}

// ------------------------------------------------------------------ pack --
// A thread has 32 columns of a row; the group's largest |w| meets over its
// one, two or four threads (neighbours: a wave holds whole groups).  10576 x 2560:
// bf16 17.8 us (floor 11), fp32 20.5 (20).
template <typename In>
__global__ __launch_bounds__(256) void s6_q4_pack_kernel(const In* w, int64_t stride, uint8_t* codes, uint16_t* scales,
                                                         int64_t base, int64_t total, int64_t per, int group) {
  const int64_t i = base + (int64_t)blockIdx.x * 256 + threadIdx.x;
  const bool on = i < total;
  const int64_t row = on ? i / per : 0, at = on ? i - row * per : 0;
  const In* p = w + row * stride + at * 32;
  float v[32];
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    v[j] = to_f32(p[j]);
    const uint32_t m = __float_as_uint(v[j]) & 0x7fffffffu;  // a NaN is above all
    top = m > top ? m : top;
  }
  for (int d = 1; d < group / 32; d *= 2) {
    const uint32_t o = __shfl_xor(top, d);
    top = o > top ? o : top;
  }
  const uint16_t sb = from_f32<uint16_t>(__uint_as_float(top) / 6.0f);
  const float s = to_f32(sb);
  uint32_t c[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t o = 0;
    if (s > 0.0f) {
      o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[8 * j] / s, v[8 * j + 1] / s, 1.0f, 0);
      o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[8 * j + 2] / s, v[8 * j + 3] / s, 1.0f, 1);
      o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[8 * j + 4] / s, v[8 * j + 5] / s, 1.0f, 2);
      o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[8 * j + 6] / s, v[8 * j + 7] / s, 1.0f, 3);
    }
    c[j] = o;
  }
  if (!on) return;
  *reinterpret_cast<uint4*>(codes + i * 16) = make_uint4(c[0], c[1], c[2], c[3]);
  if (at % (group / 32) == 0) scales[i / (group / 32)] = sb;
}

// ------------------------------------------------------------------ host --
constexpr int64_t kMaxGrid = 1 << 22;  // workgroups of a launch in x (threads below 2^32)

int check_q4(int64_t rows, int64_t inner, int64_t outer, int64_t group, int64_t stride) {
  if (rows < 0 || outer < 0 || inner < 1 || stride < 0) return S6_ERR_SHAPE;
  if (group != 32 && group != 64 && group != 128) return S6_ERR_UNSUPPORTED;
  if (inner % group || inner > kMaxStride || outer > INT32_MAX || (rows > 1 && stride < inner)) return S6_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(outer, inner, &t) || !mul_ok(t, 8, &t) || !mul_ok(rows, stride, &t) || !mul_ok(t, 8, &t) ||
      !mul_ok(rows, outer, &t) || !mul_ok(t, 64, &t))
    return S6_ERR_SHAPE;
  return S6_OK;
}

// Most rows of the first kernel, which reads x again for every 16 weight rows.
// With it and with the second, us: fp32 of 5120 to 2560, groups of 32, 6 rows 11.8
// and 10.5, 16 14.8 and 11.7, of 2560 to 10576 6 rows 13.9 and 14.2; bf16 of 2560 to
// 10576, 8 rows 8.9 and 10.5, 16 11.4 both, 24 (two tiles of rows) 16 and 13; of 8192
// to 3305, where the first loses sooner, 16 rows 13.6 and 17 with the second 12.4.
int64_t few_rows(int x_dtype) { return x_dtype == S6_F32 ? 6 : kFewRows; }
constexpr int64_t kLaunchRows = 32768;    // most rows of a launch of the second

// Rows of x to a workgroup of the second kernel.  Measured with 32 and with 64, us:
// 64 bf16 rows of 2560 to 10576: 16 and 21; 128 of 5120 to 2560, groups of 32: 18
// and 21; 256 of 2560 to 10576: 34 and 29 (fp32 rows, three parts: 32, for the
// LDS).  96 where a CU then has fewer rows in turn.  With 64 and with 96, groups of
// 32: 256 of 2560 to 10576 (128 rows in turn and 96) 38 and 27, 384 (128 and 192)
// 39 and 48, 1024 of 5120 to 2560 (128 and 96) 67 and 46.
int64_t many_rows(int64_t rows, int64_t outer, int x_dtype) {
  if (rows <= 128 || x_dtype == S6_F32) return 32;
  const int64_t tiles = (outer + kBN - 1) / kBN, cus = cu_count();
  auto in_turn = [&](int64_t bm) { return (tiles * ((rows + bm - 1) / bm) + cus - 1) / cus * bm; };
  return in_turn(96) < in_turn(64) ? 96 : 64;
}

// Slices of the columns for the second kernel: a workgroup per CU where there
// are columns for it, of at least four blocks each.  They cost a pass over their
// sums.
int64_t slices_of(int64_t rows, int64_t inner, int64_t outer, int x_dtype, int64_t* slice) {
  const int64_t nb = (inner + kBlk - 1) / kBlk, n = rows < kLaunchRows ? rows : kLaunchRows, bm = many_rows(n, outer, x_dtype);
  const int64_t tiles = ((outer + kBN - 1) / kBN) * ((n + bm - 1) / bm);
  int64_t s = cu_count() / (tiles > 0 ? tiles : 1);
  if (s > nb / 4) s = nb / 4;
  if (s < 1) s = 1;
  *slice = (nb + s - 1) / s;
  return (nb + *slice - 1) / *slice;
}

template <typename XT, bool FINE, bool XV, typename YT>
int launch_few(Q4Args a, hipStream_t st) {
  const int64_t nb = (a.inner + kBlk - 1) / kBlk, tiles = (a.outer + 15) / 16;
  // waves: as many as load the columns at once, four blocks each
  int64_t W = (nb + 3) / 4;
  if (W > 16) W = 16;
  const size_t lds = (size_t)(W - 1) * 64 * sizeof(f32x4);
  for (a.base = 0; a.base < tiles; a.base += kMaxGrid) {
    const dim3 grid((unsigned)(tiles - a.base < kMaxGrid ? tiles - a.base : kMaxGrid));
    hipLaunchKernelGGL((s6_q4_few_kernel<XT, FINE, XV, YT>), grid, dim3(64 * (unsigned)W), lds, st, a);
    S6_HIP(hipGetLastError(), "s6_q4_few_kernel launch");
  }
  return S6_OK;
}
template <typename XT, int BM, bool FINE, bool XV, typename YT>
int launch_many(Q4Args a, int64_t slices, hipStream_t st) {
  const auto kern = s6_q4_many_kernel<XT, BM, FINE, XV, YT>;
  constexpr size_t lds = many_lds(BM, sizeof(XT) == 4 ? 3 : 1);
  if constexpr (lds > 65536)
    S6_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds),
           "s6_q4_many_kernel LDS size");
  const int64_t tiles = (a.outer + kBN - 1) / kBN;
  for (a.base = 0; a.base < tiles; a.base += kMaxGrid) {
    const dim3 grid((unsigned)(tiles - a.base < kMaxGrid ? tiles - a.base : kMaxGrid), (unsigned)((a.rows + BM - 1) / BM),
                    (unsigned)slices);
    hipLaunchKernelGGL(kern, grid, dim3(512), lds, st, a);
    S6_HIP(hipGetLastError(), "s6_q4_many_kernel launch");
  }
  if (slices > 1) {
    hipLaunchKernelGGL(s6_q4_join_kernel<YT>, dim3((unsigned)((a.outer + 255) / 256), (unsigned)a.rows), dim3(256), 0, st,
                       a, (int)slices);
    S6_HIP(hipGetLastError(), "s6_q4_join_kernel launch");
  }
  return S6_OK;
}
template <typename XT, bool FINE, bool XV, typename YT>
int launch_rows(const Q4Args& a, hipStream_t st) {
  constexpr int dt = sizeof(XT) == 4 ? S6_F32 : sizeof(XT) == 2 ? S6_BF16 : S6_E4M3;
  if (a.rows <= few_rows(dt)) return launch_few<XT, FINE, XV, YT>(a, st);
  int64_t slice;
  const int64_t slices = slices_of(a.rows, a.inner, a.outer, dt, &slice);
  const int64_t bm = many_rows(a.rows < kLaunchRows ? a.rows : kLaunchRows, a.outer, dt);
  for (int64_t r = 0; r < a.rows; r += kLaunchRows) {
    Q4Args b = a;
    b.rows = a.rows - r < kLaunchRows ? a.rows - r : kLaunchRows;
    b.x = static_cast<const XT*>(a.x) + r * a.x_stride;
    b.x_scale = a.x_scale ? a.x_scale + r : nullptr;
    b.y = static_cast<YT*>(a.y) + r * a.outer;
    b.slice = (int)slice;
    if (slices == 1) b.parts = nullptr;
    int rc;
    if (bm == 32) {
      rc = launch_many<XT, 32, FINE, XV, YT>(b, slices, st);
    } else {
      if constexpr (sizeof(XT) == 4) return S6_ERR_UNSUPPORTED;  // not reached: many_rows
      else rc = bm == 64 ? launch_many<XT, 64, FINE, XV, YT>(b, slices, st) : launch_many<XT, 96, FINE, XV, YT>(b, slices, st);
    }
    if (rc) return rc;
  }
  return S6_OK;
}
template <typename XT, typename YT>
int launch_q4(Q4Args a, bool vec, hipStream_t st) {
  a.up = 1.0f / kDown<XT>;
  if (a.fine == 0) return vec ? launch_rows<XT, false, true, YT>(a, st) : launch_rows<XT, false, false, YT>(a, st);
  return vec ? launch_rows<XT, true, true, YT>(a, st) : launch_rows<XT, true, false, YT>(a, st);
}

size_t q4_ws(int64_t rows, int64_t inner, int64_t outer, int x_dtype) {
  if (rows <= few_rows(x_dtype) || outer == 0) return 0;
  int64_t slice;
  const int64_t s = slices_of(rows, inner, outer, x_dtype, &slice);
  const int64_t n = rows < kLaunchRows ? rows : kLaunchRows;
  return s > 1 ? up256((size_t)s * n * outer * sizeof(float)) : 0;
}

}  // namespace

}  // namespace s6i

using namespace s6i;

extern "C" {

int s6_q4_pack(int64_t outer, int64_t inner, int64_t group, int in_dtype, const void* w, int64_t w_stride,
               void* codes, void* scales, void* stream) {
  if (in_dtype != S6_F32 && in_dtype != S6_BF16) return S6_ERR_DTYPE;
  const int rc = check_q4(outer, inner, outer, group, w_stride);
  if (rc) return rc;
  if (outer == 0) return S6_OK;
  if (!w || !codes || !scales) return S6_ERR_NULL;
  if (!aligned(w, in_dtype == S6_BF16 ? 2 : 4) || !aligned(codes, 16) || !aligned(scales, 2)) return S6_ERR_ALIGN;
  const int64_t per = inner / 32, total = outer * per;
  hipStream_t st = static_cast<hipStream_t>(stream);
  for (int64_t base = 0; base < total; base += kMaxGrid * 256) {
    const int64_t blocks = (total - base + 255) / 256;
    const dim3 grid((unsigned)(blocks < kMaxGrid ? blocks : kMaxGrid));
    if (in_dtype == S6_BF16)
      hipLaunchKernelGGL(s6_q4_pack_kernel<uint16_t>, grid, dim3(256), 0, st, static_cast<const uint16_t*>(w), w_stride,
                         static_cast<uint8_t*>(codes), static_cast<uint16_t*>(scales), base, total, per, (int)group);
    else
      hipLaunchKernelGGL(s6_q4_pack_kernel<float>, grid, dim3(256), 0, st, static_cast<const float*>(w), w_stride,
                         static_cast<uint8_t*>(codes), static_cast<uint16_t*>(scales), base, total, per, (int)group);
    S6_HIP(hipGetLastError(), "s6_q4_pack_kernel launch");
  }
  return S6_OK;
}

int s6_q4_linear_workspace_size(int64_t rows, int64_t inner, int64_t outer, int64_t group, int x_dtype,
                                size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  if (x_dtype != S6_F32 && x_dtype != S6_BF16 && x_dtype != S6_E4M3) return S6_ERR_DTYPE;
  const int rc = check_q4(rows, inner, outer, group, inner);
  if (rc) return rc;
  *bytes = q4_ws(rows, inner, outer, x_dtype);
  return S6_OK;
}

int s6_q4_linear(int64_t rows, int64_t inner, int64_t outer, int64_t group, int x_dtype, int y_dtype, const void* x,
                 int64_t x_stride, const float* x_scale, const void* codes, const void* scales, void* y,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (x_dtype != S6_F32 && x_dtype != S6_BF16 && x_dtype != S6_E4M3) return S6_ERR_DTYPE;
  if (y_dtype != S6_F32 && y_dtype != S6_BF16) return S6_ERR_DTYPE;
  const int rc = check_q4(rows, inner, outer, group, x_stride);
  if (rc) return rc;
  if (rows > 1 && x_stride > kMaxStride) return S6_ERR_SHAPE;
  if (x_scale && x_dtype != S6_E4M3) return S6_ERR_UNSUPPORTED;
  if (rows == 0 || outer == 0) return S6_OK;
  if (!x || !codes || !scales || !y) return S6_ERR_NULL;
  const size_t xsz = x_dtype == S6_F32 ? 4 : x_dtype == S6_BF16 ? 2 : 1, ysz = y_dtype == S6_BF16 ? 2 : 4;
  if (!aligned(x, xsz) || !aligned(y, ysz) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(x_scale, 4))
    return S6_ERR_ALIGN;
  const size_t need = q4_ws(rows, inner, outer, x_dtype);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return S6_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return S6_ERR_ALIGN;
  }
  Q4Args a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.x_scale = x_scale; a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint16_t*>(scales); a.y = y;
  a.rows = rows; a.inner = (int)inner; a.outer = outer; a.x_stride = x_stride;
  a.fine = group == 128 ? 0 : group == 64 ? 1 : 2; a.ngroups = (int)(inner / group);
  a.parts = static_cast<float*>(workspace);
  a.wide = aligned(y, 16) && (outer * (int64_t)ysz) % 16 == 0;
  const bool vec = aligned(x, 16) && (x_stride * (int64_t)xsz) % 16 == 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (x_dtype == S6_F32)
    return y_dtype == S6_F32 ? launch_q4<float, float>(a, vec, st) : launch_q4<float, uint16_t>(a, vec, st);
  if (x_dtype == S6_BF16)
    return y_dtype == S6_F32 ? launch_q4<uint16_t, float>(a, vec, st) : launch_q4<uint16_t, uint16_t>(a, vec, st);
  return y_dtype == S6_F32 ? launch_q4<uint8_t, float>(a, vec, st) : launch_q4<uint8_t, uint16_t>(a, vec, st);
}

}  // extern "C"
