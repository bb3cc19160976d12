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
#include "s6_q4.h"

#include "block_internal.h"

namespace s6i {

namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

struct Q4Args {
  const void* x;
  const float* x_scale;
  const uint8_t* codes;
  const uint16_t* scales;
  void* y;
  int64_t rows, inner, outer, x_stride;
  int group;      // columns of a scale
  int ngroups;    // inner / group
  int64_t base;   // first tile of weight rows of the launch
};

// Eight codes as bf16.
__device__ __forceinline__ bf16x8 values8(uint32_t c) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2);
  const bf16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3);
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

// Eight consecutive values of x as loaded, and as bf16 parts whose sum they are.
template <typename XT, bool XV>
struct X8 {
  static constexpr int kParts = sizeof(XT) == 4 ? 3 : 1;
  alignas(16) XT e[8];
  __device__ __forceinline__ void load(const XT* p) {
    if constexpr (XV && sizeof(XT) == 1) {
      *reinterpret_cast<uint2*>(e) = *reinterpret_cast<const uint2*>(p);
    } else if constexpr (XV) {
#pragma unroll
      for (int i = 0; i < (int)sizeof(XT) / 2; ++i)
        reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = p[i];
    }
  }
  __device__ __forceinline__ void get(bf16x8 (&o)[kParts]) const {
    if constexpr (sizeof(XT) == 4) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        // what a part leaves is exact; a value that is not finite stays in the first
        const __bf16 h = (__bf16)e[i];
        float r = e[i] - (float)h;
        r = __builtin_fabsf(r) < __builtin_inff() ? r : 0.0f;
        const __bf16 m = (__bf16)r;
        o[0][i] = h;
        o[1][i] = m;
        o[2][i] = (__bf16)(r - (float)m);
      }
    } else if constexpr (sizeof(XT) == 2) {
      o[0] = __builtin_bit_cast(bf16x8, *reinterpret_cast<const uint4*>(e));
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(e);
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

// Few rows.  A workgroup has 16 weight rows and 16 NT rows of x; its W waves
// take the blocks of columns in turn and add their sums in LDS in a fixed order.  Lane
// l holds weight row l % 16 (operand), x row l % 16, and the sums of weight
// rows 4 (l / 16) to + 3.  FINE: groups of 32 or 64 columns: the codes are
// transposed so that an instruction's 32 columns lie in one group (else its
// columns are four runs of 8 from the block, all in the block's group).
template <typename XT, int NT, bool FINE, bool XV, typename YT>
__global__ __launch_bounds__(1024) void s6_q4_few_kernel(Q4Args a) {
  extern __shared__ float part[];  // (W - 1, NT, 64, 4)
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), W = blockDim.x >> 6;
  const int i = lane & 15, q = lane >> 4;
  const int64_t n0 = (a.base + blockIdx.x) * 16, t0 = (int64_t)blockIdx.y * (16 * NT);
  const int64_t n = n0 + i < a.outer ? n0 + i : a.outer - 1;
  const uint8_t* wrow = a.codes + n * (a.inner >> 1);
  const XT* xrow[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    const int64_t t = t0 + 16 * u + i;
    xrow[u] = static_cast<const XT*>(a.x) + (t < a.rows ? t : a.rows - 1) * a.x_stride;
  }
  const uint16_t* srow[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int64_t m = n0 + 4 * q + r;
    srow[r] = a.scales + (m < a.outer ? m : a.outer - 1) * a.ngroups;
  }
  f32x4 sum[NT];
#pragma unroll
  for (int u = 0; u < NT; ++u) sum[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  const int64_t nb = (a.inner + kBlk - 1) / kBlk;
  using X = X8<XT, XV>;
  for (int64_t b = wave; b < nb; b += W) {
    const int64_t k0 = b * kBlk;
    uint32_t c[4] = {0, 0, 0, 0};
    if (!FINE || k0 + 32 * q < a.inner) {
      const uint4 v = *reinterpret_cast<const uint4*>(wrow + (k0 >> 1) + 16 * q);
      c[0] = v.x; c[1] = v.y; c[2] = v.z; c[3] = v.w;
    }
    if constexpr (FINE) transpose4(c);
    f32x4 acc[NT];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (FINE && k0 + 32 * j >= a.inner) break;
      const int64_t k = k0 + (FINE ? 32 * j + 8 * q : 32 * q + 8 * j);
      const bool begin = FINE ? (k0 + 32 * j) % a.group == 0 : j == 0;
      const bool end = FINE ? (k0 + 32 * (j + 1)) % a.group == 0 : j == 3;
      const bf16x8 w = values8(c[j]);
#pragma unroll
      for (int u = 0; u < NT; ++u) {
        X xr;
        bf16x8 xp[X::kParts];
        xr.load(xrow[u] + k);
        xr.get(xp);
        if (begin) acc[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int p = X::kParts - 1; p >= 0; --p)
          acc[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, xp[p], acc[u], 0, 0, 0);
      }
      if (end) {
        const int64_t g = FINE ? (k0 + 32 * j) / a.group : b;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float s = to_f32(srow[r][g]);
#pragma unroll
          for (int u = 0; u < NT; ++u) sum[u][r] = __builtin_fmaf(s, acc[u][r], sum[u][r]);
        }
      }
    }
  }
  f32x4* parts = reinterpret_cast<f32x4*>(part);
  if (wave > 0) {
#pragma unroll
    for (int u = 0; u < NT; ++u) parts[((wave - 1) * NT + u) * 64 + lane] = sum[u];
  }
  __syncthreads();
  if (wave > 0) return;
#pragma unroll
  for (int u = 0; u < NT; ++u) {
    for (int w = 0; w + 1 < W; ++w) sum[u] += parts[(w * NT + u) * 64 + lane];
    const int64_t t = t0 + 16 * u + i;
    if (t >= a.rows) continue;
    const float xs = a.x_scale ? a.x_scale[t] : 1.0f;
    YT* y = static_cast<YT*>(a.y) + t * a.outer;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n0 + 4 * q + r < a.outer) y[n0 + 4 * q + r] = from_f32<YT>(sum[u][r] * xs);
  }
}

// ------------------------------------------------------------------ pack --
// A thread has 32 columns of a row; the group's largest |w| meets over its
// one, two or four threads (neighbours: a wave holds whole groups).
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
  if (inner % group || inner > (1 << 28) || outer > INT32_MAX || (rows > 1 && stride < inner)) return S6_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(outer, inner, &t) || !mul_ok(t, 8, &t) || !mul_ok(rows, stride, &t) || !mul_ok(t, 8, &t) ||
      !mul_ok(rows, outer, &t) || !mul_ok(t, 64, &t))
    return S6_ERR_SHAPE;
  return S6_OK;
}

template <typename XT, int NT, bool FINE, bool XV, typename YT>
int launch_few(Q4Args a, hipStream_t st) {
  const int64_t nb = (a.inner + kBlk - 1) / kBlk, tiles = (a.outer + 15) / 16;
  const int64_t ty = (a.rows + 16 * NT - 1) / (16 * NT);
  // waves: about five blocks each
  const int W = nb > 40 ? 16 : nb > 20 ? 8 : nb > 2 ? 4 : nb > 1 ? 2 : 1;
  const size_t lds = (size_t)(W - 1) * NT * 64 * sizeof(f32x4);
  for (a.base = 0; a.base < tiles; a.base += kMaxGrid) {
    const dim3 grid((unsigned)(tiles - a.base < kMaxGrid ? tiles - a.base : kMaxGrid), (unsigned)ty);
    hipLaunchKernelGGL((s6_q4_few_kernel<XT, NT, FINE, XV, YT>), grid, dim3(64 * W), lds, st, a);
    S6_HIP(hipGetLastError(), "s6_q4_few_kernel launch");
  }
  return S6_OK;
}
template <typename XT, bool FINE, bool XV, typename YT>
int launch_rows(Q4Args a, hipStream_t st) {
  // at most 65535 tiles of rows a launch
  const int64_t rows = a.rows, step = 65535 * 16;
  for (int64_t r = 0; r < rows; r += step) {
    Q4Args b = a;
    b.rows = rows - r < step ? rows - r : step;
    b.x = static_cast<const XT*>(a.x) + r * a.x_stride;
    b.x_scale = a.x_scale ? a.x_scale + r : nullptr;
    b.y = static_cast<YT*>(a.y) + r * a.outer;
    const int rc = b.rows <= 16 ? launch_few<XT, 1, FINE, XV, YT>(b, st)
                   : b.rows <= 32 ? launch_few<XT, 2, FINE, XV, YT>(b, st)
                                  : launch_few<XT, 4, FINE, XV, YT>(b, st);
    if (rc) return rc;
  }
  return S6_OK;
}
template <typename XT, typename YT>
int launch_q4(const Q4Args& a, bool vec, hipStream_t st) {
  if (a.group == 128) return vec ? launch_rows<XT, false, true, YT>(a, st) : launch_rows<XT, false, false, YT>(a, st);
  return vec ? launch_rows<XT, true, true, YT>(a, st) : launch_rows<XT, true, false, YT>(a, st);
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
  *bytes = 0;
  return S6_OK;
}

int s6_q4_linear(int64_t rows, int64_t inner, int64_t outer, int64_t group, int x_dtype, int y_dtype, const void* x,
                 int64_t x_stride, const float* x_scale, const void* codes, const void* scales, void* y,
                 void* workspace, size_t workspace_bytes, void* stream) {
  if (x_dtype != S6_F32 && x_dtype != S6_BF16 && x_dtype != S6_E4M3) return S6_ERR_DTYPE;
  if (y_dtype != S6_F32 && y_dtype != S6_BF16) return S6_ERR_DTYPE;
  const int rc = check_q4(rows, inner, outer, group, x_stride);
  if (rc) return rc;
  if (x_scale && x_dtype != S6_E4M3) return S6_ERR_UNSUPPORTED;
  if (rows == 0 || outer == 0) return S6_OK;
  if (!x || !codes || !scales || !y) return S6_ERR_NULL;
  const size_t xsz = x_dtype == S6_F32 ? 4 : x_dtype == S6_BF16 ? 2 : 1, ysz = y_dtype == S6_BF16 ? 2 : 4;
  if (!aligned(x, xsz) || !aligned(y, ysz) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(x_scale, 4))
    return S6_ERR_ALIGN;
  (void)workspace; (void)workspace_bytes;
  Q4Args a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.x_scale = x_scale; a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint16_t*>(scales); a.y = y;
  a.rows = rows; a.inner = inner; a.outer = outer; a.x_stride = x_stride;
  a.group = (int)group; a.ngroups = (int)(inner / group);
  const bool vec = aligned(x, 16) && (x_stride * (int64_t)xsz) % 16 == 0;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (x_dtype == S6_F32)
    return y_dtype == S6_F32 ? launch_q4<float, float>(a, vec, st) : launch_q4<float, uint16_t>(a, vec, st);
  if (x_dtype == S6_BF16)
    return y_dtype == S6_F32 ? launch_q4<uint16_t, float>(a, vec, st) : launch_q4<uint16_t, uint16_t>(a, vec, st);
  return y_dtype == S6_F32 ? launch_q4<uint8_t, float>(a, vec, st) : launch_q4<uint8_t, uint16_t>(a, vec, st);
}

}  // extern "C"
