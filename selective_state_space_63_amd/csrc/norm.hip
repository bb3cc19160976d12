// norm.hip -- the norms around a block (include/s6_block.h): the residual
// add, residual scale and RMS norm before it (s6_add_norm_*), the SiLU gate
// and grouped RMS norm after its scan (s6_gated_norm_*), and their gradients.
//
// Per row (of a group) u of d values, i = 1 / sqrt(mean(u^2) + eps):
//   out = u i w
//   du_k = i (dh_k - u_k i m),  dh = dout w,  m = (i / d) sum_k dh_k u_k
//   dw_k = sum over rows of dout_k u_k i
// Both sums of the backward, sum u^2 and sum dh u, need the inputs alone, so
// each direction reads its inputs once, keeps them in registers, adds across
// the row's threads once and writes its outputs: the forward is bound by HBM,
// the backward by the few rows that its registers let a CU hold at once (see
// norm_plan).  Sums and statistics are fp32.
//
// Layout: a row is a workgroup's (as many waves as hold it), or, for narrow
// rows, a wave's with four rows per workgroup.  Each thread keeps K pieces of V
// consecutive values in registers (V = 8: 16-byte accesses; V = 1 where a
// width, stride or pointer does not allow them); rows wider than that read the
// rest again in the second phase.  A thread keeps its columns over the rows it
// walks, so weights are read once per thread and the column sums (dw, dgamma)
// stay in registers until the end; the row walkers' parts are then added in a
// fixed order by s6_norm_colsum.  The next row's loads are issued before the
// current row's sums meet.
//
// Training passes (forward, backward and column sums), bf16: 16384 rows of
// 2560 with an fp32 residual 271 us (4.6 TB/s), gated 16384 rows of 5120 325 us
// (4.1 TB/s), of which the backward kernels 158 and 215 us (4.7 and 3.9 TB/s);
// 256 rows of 2560: 3.7 us of kernel, 10.6 us with the call.
#include "block_internal.h"
#include "s6_q4.h"

namespace s6i {

namespace {

constexpr int kMaxT = 1024;        // threads of a workgroup
constexpr float kTopQ8 = 448.0f;   // largest e4m3 value
constexpr int64_t kParts = 1024;   // most row walkers where column sums are taken (each leaves a part)

struct NormArgs {
  int64_t rows, dim, gd;        // gd: width of a group (dim for the add norm)
  const void* a;                // x (add), y (gate)
  int64_t a_stride;
  const void* b;                // residual (add), z (gate); nullable
  int64_t b_stride;
  const void* dout;
  const void* dres;             // dresidual_out (add), nullable
  const void* res;              // residual_out (add backward)
  const float* w;
  const float* gamma;           // nullable
  float scale, eps;
  int after;                    // gate after the norm
  void* o1;                     // out / dx / dy
  void* o2;                     // residual_out / dresidual / dz
  float* dw;                    // parts (walkers, dim), nullable
  float* dg;                    // parts (walkers, dim), nullable
  float* row_scale;             // scales of an 8-bit output
};

// V values of a row as loaded.
template <typename T, int V>
struct Raw {
  T e[V];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      e[0] = *p;
    } else {
#pragma unroll
      for (int i = 0; i < (int)(V * sizeof(T)) / 16; ++i)
        reinterpret_cast<uint4*>(e)[i] = reinterpret_cast<const uint4*>(p)[i];
    }
  }
  __device__ __forceinline__ void get(float (&f)[V]) const {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = to_f32(e[j]);
  }
  // What is formed from the values before is formed again after this, instead
  // of being kept in registers as floats.
  __device__ __forceinline__ void again() {
    if constexpr (V > 1) {
      uint32_t w[V * sizeof(T) / 4];
      __builtin_memcpy(w, e, sizeof(e));
#pragma unroll
      for (int i = 0; i < (int)(V * sizeof(T)) / 4; ++i) asm volatile("" : "+v"(w[i]));
      __builtin_memcpy(e, w, sizeof(e));
    }
  }
};

__device__ __forceinline__ float sigmoid_f(float z) { return fast_rcp(1.0f + fast_exp2(-z * kLog2e)); }

// The rows that a thread walks: wk, wk + nw, ...; every walker of a workgroup
// makes the same number of turns (barriers), masked past the end.  t of tpr:
// the thread in its row.
struct Walk {
  int64_t wk, nw, turns;
  int t, tpr;
};
template <bool MULTI>
__device__ __forceinline__ Walk walk_of(int64_t rows) {
  Walk o;
  const int per = MULTI ? 4 : 1;
  o.tpr = MULTI ? 64 : (int)blockDim.x;
  o.nw = (int64_t)gridDim.x * per;
  o.wk = (int64_t)blockIdx.x * per + (MULTI ? threadIdx.x >> 6 : 0);
  o.turns = (rows + o.nw - 1) / o.nw;
  o.t = MULTI ? threadIdx.x & 63 : threadIdx.x;
  return o;
}

// Sums of two values over the threads of a row.  The waves of a workgroup
// meet in LDS; the buffer alternates between two halves, so one barrier per
// row is enough (a wave writes half i again only after the barrier of half
// i + 1, which every wave reaches after reading half i).
template <bool MULTI>
__device__ __forceinline__ void row_sum2(float& s, float& t, float (*buf)[2][kMaxT / 64], int par) {
  s = wave_sum(s);
  t = wave_sum(t);
  if constexpr (!MULTI) {
    const int w = threadIdx.x >> 6, n = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) { buf[par][0][w] = s; buf[par][1][w] = t; }
    __syncthreads();
    s = t = 0.0f;
    for (int i = 0; i < n; ++i) { s += buf[par][0][i]; t += buf[par][1][i]; }
  }
}

// ------------------------------------------------------------- add norm --
template <typename In, typename Res, int V, int K, bool MULTI, bool WIDE>
__global__ __launch_bounds__(K == 2 ? 512 : kMaxT) void s6_add_norm_kernel(NormArgs a) {
  __shared__ float buf[2][2][kMaxT / 64];
  const Walk wk = walk_of<MULTI>(a.rows);
  const int64_t np = (a.dim + V - 1) / V;  // pieces of a row
  const float inv_d = 1.0f / (float)a.dim;
  float w[K][V], ga[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t i = (int64_t)k * wk.tpr + wk.t;
#pragma unroll
    for (int j = 0; j < V; ++j) ga[k][j] = a.scale;
    if (i < np) {
      load_vec<float, V>(a.w + i * V, w[k]);
      if (a.gamma) {
        load_vec<float, V>(a.gamma + i * V, ga[k]);
#pragma unroll
        for (int j = 0; j < V; ++j) ga[k][j] *= a.scale;
      }
    }
  }
  Raw<In, V> xr[K];
  Raw<Res, V> rr[K];
  auto issue = [&](int64_t row) {
    if (row >= a.rows) return;
    const In* x = static_cast<const In*>(a.a) + row * a.a_stride;
    const Res* r = static_cast<const Res*>(a.b) + row * a.dim;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (i < np) {
        xr[k].load(x + i * V);
        if (a.b) rr[k].load(r + i * V);
      }
    }
  };
  issue(wk.wk);
  for (int64_t q = 0; q < wk.turns; ++q) {
    const int64_t row = q * wk.nw + wk.wk;
    const bool on = row < a.rows;
    const In* x = static_cast<const In*>(a.a) + row * a.a_stride;
    const Res* r = a.b ? static_cast<const Res*>(a.b) + row * a.dim : nullptr;
    In* out = static_cast<In*>(a.o1) + row * a.dim;
    Res* ro = static_cast<Res*>(a.o2) + row * a.dim;
    float u[K][V];
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
        float rv[V];
        xr[k].get(u[k]);
        if (r) rr[k].get(rv);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          u[k][j] = r ? __builtin_fmaf(ga[k][j], u[k][j], rv[j]) : ga[k][j] * u[k][j];
          s = __builtin_fmaf(u[k][j], u[k][j], s);
        }
        store_vec<Res, V>(ro + i * V, u[k]);
      }
    }
    issue(row + wk.nw);
    // a piece past the registers: r' is formed again for out, from x and the
    // residual, so it is stored in the second phase (residual_out may be the
    // residual's buffer)
    auto wide = [&](int64_t i, float (&v)[V]) {
      float rv[V], gg[V];
      load_vec<In, V>(x + i * V, v);
      if (r) load_vec<Res, V>(r + i * V, rv);
      if (a.gamma) load_vec<float, V>(a.gamma + i * V, gg);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g = a.gamma ? gg[j] * a.scale : a.scale;
        v[j] = r ? __builtin_fmaf(g, v[j], rv[j]) : g * v[j];
      }
    };
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float v[V];
      wide(i, v);
#pragma unroll
      for (int j = 0; j < V; ++j) s = __builtin_fmaf(v[j], v[j], s);
    }
    row_sum2<MULTI>(s, unused, buf, (int)(q & 1));
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_d, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
#pragma unroll
        for (int j = 0; j < V; ++j) u[k][j] = u[k][j] * inv * w[k][j];
        store_vec<In, V>(out + i * V, u[k]);
      }
    }
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float v[V], ww[V];
      wide(i, v);
      load_vec<float, V>(a.w + i * V, ww);
      store_vec<Res, V>(ro + i * V, v);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = v[j] * inv * ww[j];
      store_vec<In, V>(out + i * V, v);
    }
  }
}

// -------------------------------------------------- add norm, 8-bit output --
// The largest of unsigned values over the threads of a row, as row_sum2; as
// bits of |v|, an infinity is above all numbers and a NaN above that.
template <bool MULTI>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t (*buf)[kMaxT / 64], int par) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const uint32_t o = __shfl_xor(m, d);
    m = o > m ? o : m;
  }
  if constexpr (!MULTI) {
    const int w = threadIdx.x >> 6, n = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0) buf[par][w] = m;
    __syncthreads();
    m = 0;
    for (int i = 0; i < n; ++i) m = buf[par][i] > m ? buf[par][i] : m;
  }
  return m;
}

// v / unit with f = 1 / unit but for a rounding or two: what the product lacks of v
// corrects it, so a value between two codes goes to the one that the quotient does.
__device__ __forceinline__ float over(float v, float unit, float f) {
  const float q = v * f;
  return __builtin_fmaf(__builtin_fmaf(-q, unit, v), f, q);
}
// V values over unit as e4m3; all NaN where nan is set.
template <int V>
__device__ __forceinline__ void store_q8(uint8_t* p, const float (&v)[V], float unit, float f, bool nan) {
  if constexpr (V == 1) {
    *p = nan ? 0x7f : (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(over(v[0], unit, f), 0.0f, 0, false);
  } else {
    uint32_t o[V / 4];
#pragma unroll
    for (int i = 0; i < V / 4; ++i) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(over(v[4 * i], unit, f), over(v[4 * i + 1], unit, f), 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(over(v[4 * i + 2], unit, f), over(v[4 * i + 3], unit, f), w, true);
      o[i] = nan ? 0x7f7f7f7fu : (uint32_t)w;
    }
    if constexpr (V == 8) *reinterpret_cast<uint2*>(p) = make_uint2(o[0], o[1]);
  }
}

// As s6_add_norm_kernel, with the row's largest output found before any is
// stored: the outputs stay in registers, or are formed again past them.
// 16384 bf16 rows of 2560 with an fp32 residual: 98 us (4.7 TB/s, floor 74), bound
// by HBM; 256 rows: 4.3 us.  Stores past the caches took 88 us where these took
// 104, but a sum of the codes and an addition to the residual right after took
// longer by more (262 us for 255 in all); not timed where a layer lies between.
// Six waves per SIMD where a thread has one bf16 piece of a row: 16384 x 2560 98 us, with
// the five that the registers would leave 104 (fp32 would spill).
template <typename In, typename Res, int V, int K, bool MULTI, bool WIDE>
__global__ __launch_bounds__((K == 2 ? 512 : kMaxT), (V == 8 && K == 1 && sizeof(In) == 2 ? 6 : 1))
void s6_add_norm_q8_kernel(NormArgs a) {
  __shared__ float buf[2][2][kMaxT / 64], again[2][2][kMaxT / 64];
  __shared__ uint32_t mbuf[2][kMaxT / 64];
  const Walk wk = walk_of<MULTI>(a.rows);
  const int64_t np = (a.dim + V - 1) / V;
  const float inv_d = 1.0f / (float)a.dim;
  float w[K][V], ga[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t i = (int64_t)k * wk.tpr + wk.t;
#pragma unroll
    for (int j = 0; j < V; ++j) ga[k][j] = a.scale;
    if (i < np) {
      load_vec<float, V>(a.w + i * V, w[k]);
      if (a.gamma) {
        load_vec<float, V>(a.gamma + i * V, ga[k]);
#pragma unroll
        for (int j = 0; j < V; ++j) ga[k][j] *= a.scale;
      }
    }
  }
  Raw<In, V> xr[K];
  Raw<Res, V> rr[K];
  auto issue = [&](int64_t row) {
    if (row >= a.rows) return;
    const In* x = static_cast<const In*>(a.a) + row * a.a_stride;
    const Res* r = static_cast<const Res*>(a.b) + row * a.dim;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (i < np) {
        xr[k].load(x + i * V);
        if (a.b) rr[k].load(r + i * V);
      }
    }
  };
  issue(wk.wk);
  for (int64_t q = 0; q < wk.turns; ++q) {
    const int64_t row = q * wk.nw + wk.wk;
    const bool on = row < a.rows;
    const In* x = static_cast<const In*>(a.a) + row * a.a_stride;
    const Res* r = a.b ? static_cast<const Res*>(a.b) + row * a.dim : nullptr;
    uint8_t* out = static_cast<uint8_t*>(a.o1) + row * a.dim;
    Res* ro = static_cast<Res*>(a.o2) + row * a.dim;
    float u[K][V];
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
        float rv[V];
        xr[k].get(u[k]);
        if (r) rr[k].get(rv);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          u[k][j] = r ? __builtin_fmaf(ga[k][j], u[k][j], rv[j]) : ga[k][j] * u[k][j];
          s = __builtin_fmaf(u[k][j], u[k][j], s);
        }
        store_vec<Res, V>(ro + i * V, u[k]);
      }
    }
    issue(row + wk.nw);
    // a piece past the registers, formed again in each phase and stored in the last
    auto wide = [&](int64_t i, float (&v)[V]) {
      float rv[V], gg[V];
      load_vec<In, V>(x + i * V, v);
      if (r) load_vec<Res, V>(r + i * V, rv);
      if (a.gamma) load_vec<float, V>(a.gamma + i * V, gg);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g = a.gamma ? gg[j] * a.scale : a.scale;
        v[j] = r ? __builtin_fmaf(g, v[j], rv[j]) : g * v[j];
      }
    };
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float v[V];
      wide(i, v);
#pragma unroll
      for (int j = 0; j < V; ++j) s = __builtin_fmaf(v[j], v[j], s);
    }
    row_sum2<MULTI>(s, unused, buf, (int)(q & 1));
    const float mean = __builtin_fmaf(s, inv_d, a.eps);
    float inv = __builtin_amdgcn_rsqf(mean);
    if (!(s < __builtin_inff() && mean >= 0x1p-90f)) {
      // squares past the range of fp32 (the whole row sees the same sum): again,
      // of values that are not
      const float p = mean < 1.0f ? 0x1p90f : 0x1p-80f;
      s = 0.0f;
      auto square = [&](const float (&v)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) s = __builtin_fmaf(v[j] * p, v[j] * p, s);
      };
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (on && (int64_t)k * wk.tpr + wk.t < np) square(u[k]);
      for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
        float v[V];
        wide(i, v);
        square(v);
      }
      row_sum2<MULTI>(s, unused, again, (int)(q & 1));
      inv = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_d, a.eps * p * p)) * p;
    }
    uint32_t top = 0;
    auto larger = [&](const float (&v)[V]) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const uint32_t m = __float_as_uint(v[j]) & 0x7fffffffu;
        top = m > top ? m : top;
      }
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
#pragma unroll
        for (int j = 0; j < V; ++j) u[k][j] = u[k][j] * inv * w[k][j];
        larger(u[k]);
      }
    }
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float v[V], ww[V];
      wide(i, v);
      load_vec<float, V>(a.w + i * V, ww);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = v[j] * inv * ww[j];
      larger(v);
    }
    top = row_max<MULTI>(top, mbuf, (int)(q & 1));
    const bool nan = top >= 0x7f800000u;
    const float most = top < 0x0d800000u ? 0.0f : __uint_as_float(top);  // 2^-100
    const float unit = most / kTopQ8;  // 0, or its reciprocal is a normal number, too
    const float f = most > 0.0f ? fast_rcp(unit) : 0.0f;
    if (on && wk.t == 0) a.row_scale[row] = nan ? __builtin_nanf("") : unit;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) store_q8<V>(out + i * V, u[k], unit, f, nan);
    }
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float v[V], ww[V];
      wide(i, v);
      load_vec<float, V>(a.w + i * V, ww);
      store_vec<Res, V>(ro + i * V, v);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = v[j] * inv * ww[j];
      store_q8<V>(out + i * V, v, unit, f, nan);
    }
  }
}

// A column sum's part past the registers: added in memory (each walker has a
// row of its own; the first turn sets it).
template <int V>
__device__ __forceinline__ void part_add(float* p, const float (&v)[V], bool first) {
  float o[V];
  if (!first) load_vec<float, V>(p, o);
#pragma unroll
  for (int j = 0; j < V; ++j) o[j] = first ? v[j] : o[j] + v[j];
  store_vec<float, V>(p, o);
}

template <typename In, typename Res, int V, int K, bool MULTI, bool WIDE>
__global__ __launch_bounds__(K == 2 ? 512 : kMaxT) void s6_add_norm_bwd_kernel(NormArgs a) {
  __shared__ float buf[2][2][kMaxT / 64];
  const Walk wk = walk_of<MULTI>(a.rows);
  const int64_t np = (a.dim + V - 1) / V;
  const float inv_d = 1.0f / (float)a.dim;
  float w[K][V], ga[K][V], dw[K][V], dg[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t i = (int64_t)k * wk.tpr + wk.t;
#pragma unroll
    for (int j = 0; j < V; ++j) { ga[k][j] = a.scale; dw[k][j] = dg[k][j] = 0.0f; }
    if (i < np) {
      load_vec<float, V>(a.w + i * V, w[k]);
      if (a.gamma) {
        load_vec<float, V>(a.gamma + i * V, ga[k]);
#pragma unroll
        for (int j = 0; j < V; ++j) ga[k][j] *= a.scale;
      }
    }
  }
  Raw<In, V> dr_[K], xr[K];
  Raw<Res, V> ur[K], er[K];
  auto issue = [&](int64_t row) {
    if (row >= a.rows) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (i < np) {
        ur[k].load(static_cast<const Res*>(a.res) + row * a.dim + i * V);
        dr_[k].load(static_cast<const In*>(a.dout) + row * a.dim + i * V);
        if (a.dres) er[k].load(static_cast<const Res*>(a.dres) + row * a.dim + i * V);
        if (a.dg) xr[k].load(static_cast<const In*>(a.a) + row * a.a_stride + i * V);
      }
    }
  };
  issue(wk.wk);
  for (int64_t q = 0; q < wk.turns; ++q) {
    const int64_t row = q * wk.nw + wk.wk;
    const bool on = row < a.rows;
    const int64_t at = row * a.dim;
    const In* dout = static_cast<const In*>(a.dout) + at;
    const Res* res = static_cast<const Res*>(a.res) + at;
    const Res* dres = a.dres ? static_cast<const Res*>(a.dres) + at : nullptr;
    const In* x = static_cast<const In*>(a.a) + row * a.a_stride;
    In* dx = a.o1 ? static_cast<In*>(a.o1) + at : nullptr;
    Res* dr = a.o2 ? static_cast<Res*>(a.o2) + at : nullptr;
    Raw<In, V> dc[K], xc[K];
    Raw<Res, V> uc[K], ec[K];
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      dc[k] = dr_[k]; xc[k] = xr[k]; uc[k] = ur[k]; ec[k] = er[k];
      if (on && i < np) {
        float u[V], d[V];
        uc[k].get(u);
        dc[k].get(d);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          s = __builtin_fmaf(u[j], u[j], s);
          t = __builtin_fmaf(d[j] * w[k][j], u[j], t);
        }
      }
    }
    issue(row + wk.nw);
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float uu[V], dd[V], ww[V];
      load_vec<Res, V>(res + i * V, uu);
      load_vec<In, V>(dout + i * V, dd);
      load_vec<float, V>(a.w + i * V, ww);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        s = __builtin_fmaf(uu[j], uu[j], s);
        t = __builtin_fmaf(dd[j] * ww[j], uu[j], t);
      }
    }
    row_sum2<MULTI>(s, t, buf, (int)(q & 1));
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_d, a.eps));
    const float m = inv * inv * (t * inv_d);  // u i m = u m, with m including both factors i
    auto grads = [&](int64_t i, const float (&uu)[V], const float (&dd)[V], const float (&ee)[V], const float (&xx)[V],
                     const float (&ww)[V], const float (&gg)[V], float (&pw)[V], float (&pg)[V]) {
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        pw[j] = dd[j] * (uu[j] * inv);
        o[j] = inv * __builtin_fmaf(-uu[j], m, dd[j] * ww[j]) + (dres ? ee[j] : 0.0f);
      }
      if (dr) store_vec<Res, V>(dr + i * V, o);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        pg[j] = a.dg ? a.scale * (o[j] * xx[j]) : 0.0f;
        o[j] *= gg[j];
      }
      if (dx) store_vec<In, V>(dx + i * V, o);
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
        float u[V], d[V], e[V], xv[V], pw[V], pg[V];
        dc[k].again();
        uc[k].get(u);
        dc[k].get(d);
        ec[k].get(e);
        xc[k].get(xv);
        grads(i, u, d, e, xv, w[k], ga[k], pw, pg);
#pragma unroll
        for (int j = 0; j < V; ++j) { dw[k][j] += pw[j]; dg[k][j] += pg[j]; }
      }
    }
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float uu[V], dd[V], ee[V], xx[V], ww[V], gg[V], pw[V], pg[V];
      load_vec<Res, V>(res + i * V, uu);
      load_vec<In, V>(dout + i * V, dd);
      if (dres) load_vec<Res, V>(dres + i * V, ee);
      if (a.dg) load_vec<In, V>(x + i * V, xx);
      load_vec<float, V>(a.w + i * V, ww);
      if (a.gamma) load_vec<float, V>(a.gamma + i * V, gg);
#pragma unroll
      for (int j = 0; j < V; ++j) gg[j] = a.gamma ? gg[j] * a.scale : a.scale;
      grads(i, uu, dd, ee, xx, ww, gg, pw, pg);
      if (a.dw) part_add<V>(a.dw + wk.wk * a.dim + i * V, pw, q == 0);
      if (a.dg) part_add<V>(a.dg + wk.wk * a.dim + i * V, pg, q == 0);
    }
  }
  if (wk.wk >= a.rows) return;  // no row of its own: its part is not read
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t i = (int64_t)k * wk.tpr + wk.t;
    if (i < np) {
      if (a.dw) store_vec<float, V>(a.dw + wk.wk * a.dim + i * V, dw[k]);
      if (a.dg) store_vec<float, V>(a.dg + wk.wk * a.dim + i * V, dg[k]);
    }
  }
}

// ----------------------------------------------------------- gated norm --
// blockIdx.y: the group.
template <typename In, int V, int K, bool MULTI, bool WIDE>
__global__ __launch_bounds__(K == 2 ? 512 : kMaxT) void s6_gated_norm_kernel(NormArgs a) {
  __shared__ float buf[2][2][kMaxT / 64];
  const Walk wk = walk_of<MULTI>(a.rows);
  const int64_t np = (a.gd + V - 1) / V, g0 = (int64_t)blockIdx.y * a.gd;
  const float inv_d = 1.0f / (float)a.gd;
  float w[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t i = (int64_t)k * wk.tpr + wk.t;
    if (i < np) load_vec<float, V>(a.w + g0 + i * V, w[k]);
  }
  Raw<In, V> yr[K], zr[K];
  auto issue = [&](int64_t row) {
    if (row >= a.rows) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (i < np) {
        yr[k].load(static_cast<const In*>(a.a) + row * a.a_stride + g0 + i * V);
        if (a.b) zr[k].load(static_cast<const In*>(a.b) + row * a.b_stride + g0 + i * V);
      }
    }
  };
  issue(wk.wk);
  for (int64_t q = 0; q < wk.turns; ++q) {
    const int64_t row = q * wk.nw + wk.wk;
    const bool on = row < a.rows;
    const In* y = static_cast<const In*>(a.a) + row * a.a_stride + g0;
    const In* z = a.b ? static_cast<const In*>(a.b) + row * a.b_stride + g0 : nullptr;
    In* out = static_cast<In*>(a.o1) + row * a.dim + g0;
    float u[K][V], zv[K][V];
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
        yr[k].get(u[k]);
        if (z) zr[k].get(zv[k]);
      }
    }
    issue(row + wk.nw);
    // what the norm sees, and the factor applied after it
    auto gate = [&](float (&v)[V], float (&f)[V]) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float si = z ? silu(f[j]) : 1.0f;
        if (!a.after) v[j] *= si;
        f[j] = a.after ? si : 1.0f;
      }
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
        gate(u[k], zv[k]);
#pragma unroll
        for (int j = 0; j < V; ++j) s = __builtin_fmaf(u[k][j], u[k][j], s);
      }
    }
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float v[V], f[V];
      load_vec<In, V>(y + i * V, v);
      if (z) load_vec<In, V>(z + i * V, f);
      gate(v, f);
#pragma unroll
      for (int j = 0; j < V; ++j) s = __builtin_fmaf(v[j], v[j], s);
    }
    row_sum2<MULTI>(s, unused, buf, (int)(q & 1));
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_d, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
#pragma unroll
        for (int j = 0; j < V; ++j) u[k][j] = u[k][j] * inv * w[k][j] * zv[k][j];
        store_vec<In, V>(out + i * V, u[k]);
      }
    }
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float v[V], f[V], ww[V];
      load_vec<In, V>(y + i * V, v);
      if (z) load_vec<In, V>(z + i * V, f);
      load_vec<float, V>(a.w + g0 + i * V, ww);
      gate(v, f);
#pragma unroll
      for (int j = 0; j < V; ++j) v[j] = v[j] * inv * ww[j] * f[j];
      store_vec<In, V>(out + i * V, v);
    }
  }
}

template <typename In, int V, int K, bool MULTI, bool WIDE>
__global__ __launch_bounds__(K == 2 ? 512 : kMaxT) void s6_gated_norm_bwd_kernel(NormArgs a) {
  __shared__ float buf[2][2][kMaxT / 64];
  const Walk wk = walk_of<MULTI>(a.rows);
  const int64_t np = (a.gd + V - 1) / V, g0 = (int64_t)blockIdx.y * a.gd;
  const float inv_d = 1.0f / (float)a.gd;
  float w[K][V], dw[K][V];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t i = (int64_t)k * wk.tpr + wk.t;
#pragma unroll
    for (int j = 0; j < V; ++j) dw[k][j] = 0.0f;
    if (i < np) load_vec<float, V>(a.w + g0 + i * V, w[k]);
  }
  Raw<In, V> yr[K], zr[K], dr_[K];
  auto issue = [&](int64_t row) {
    if (row >= a.rows) return;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (i < np) {
        yr[k].load(static_cast<const In*>(a.a) + row * a.a_stride + g0 + i * V);
        dr_[k].load(static_cast<const In*>(a.dout) + row * a.dim + g0 + i * V);
        if (a.b) zr[k].load(static_cast<const In*>(a.b) + row * a.b_stride + g0 + i * V);
      }
    }
  };
  issue(wk.wk);
  for (int64_t q = 0; q < wk.turns; ++q) {
    const int64_t row = q * wk.nw + wk.wk;
    const bool on = row < a.rows;
    const In* y = static_cast<const In*>(a.a) + row * a.a_stride + g0;
    const In* z = a.b ? static_cast<const In*>(a.b) + row * a.b_stride + g0 : nullptr;
    const In* dout = static_cast<const In*>(a.dout) + row * a.dim + g0;
    In* dy = static_cast<In*>(a.o1) + row * a.dim + g0;
    In* dz = z ? static_cast<In*>(a.o2) + row * a.dim + g0 : nullptr;
    Raw<In, V> yc[K], zc[K], dc[K];
    float s = 0.0f, t = 0.0f;
    // u: what the norm sees; dh: the gradient of its output u i (before w)
    auto sums = [&](const float (&yy)[V], const float (&zz)[V], const float (&dd)[V], const float (&ww)[V]) {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float si = z ? silu(zz[j]) : 1.0f;
        const float u = a.after ? yy[j] : yy[j] * si;
        const float dh = (a.after ? dd[j] * si : dd[j]) * ww[j];
        s = __builtin_fmaf(u, u, s);
        t = __builtin_fmaf(dh, u, t);
      }
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      yc[k] = yr[k]; zc[k] = zr[k]; dc[k] = dr_[k];
      if (on && i < np) {
        float yv[V], zv[V], d[V];
        yc[k].get(yv);
        zc[k].get(zv);
        dc[k].get(d);
        sums(yv, zv, d, w[k]);
      }
    }
    issue(row + wk.nw);
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float yy[V], zz[V], dd[V], ww[V];
      load_vec<In, V>(y + i * V, yy);
      load_vec<In, V>(dout + i * V, dd);
      if (z) load_vec<In, V>(z + i * V, zz);
      load_vec<float, V>(a.w + g0 + i * V, ww);
      sums(yy, zz, dd, ww);
    }
    row_sum2<MULTI>(s, t, buf, (int)(q & 1));
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_d, a.eps));
    const float m = inv * inv * (t * inv_d);
    auto grads = [&](int64_t i, const float (&yy)[V], const float (&zz)[V], const float (&dd)[V], const float (&ww)[V],
                     float (&pw)[V]) {
      float oy[V], oz[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float sg = z ? sigmoid_f(zz[j]) : 1.0f;
        const float si = z ? zz[j] * sg : 1.0f;
        const float dsi = z ? __builtin_fmaf(si, 1.0f - sg, sg) : 0.0f;  // SiLU'(z)
        const float u = a.after ? yy[j] : yy[j] * si;
        const float dn = a.after ? dd[j] * si : dd[j];
        pw[j] = dn * (u * inv);
        const float du = inv * __builtin_fmaf(-u, m, dn * ww[j]);
        oy[j] = a.after ? du : du * si;
        oz[j] = (a.after ? dd[j] * (u * inv * ww[j]) : du * yy[j]) * dsi;
      }
      store_vec<In, V>(dy + i * V, oy);
      if (dz) store_vec<In, V>(dz + i * V, oz);
    };
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int64_t i = (int64_t)k * wk.tpr + wk.t;
      if (on && i < np) {
        float yv[V], zv[V], d[V], pw[V];
        yc[k].again();
        zc[k].again();
        dc[k].again();
        yc[k].get(yv);
        zc[k].get(zv);
        dc[k].get(d);
        grads(i, yv, zv, d, w[k], pw);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[k][j] += pw[j];
      }
    }
    for (int64_t i = (int64_t)K * wk.tpr + wk.t; WIDE && on && i < np; i += wk.tpr) {
      float yy[V], zz[V], dd[V], ww[V], pw[V];
      load_vec<In, V>(y + i * V, yy);
      load_vec<In, V>(dout + i * V, dd);
      if (z) load_vec<In, V>(z + i * V, zz);
      load_vec<float, V>(a.w + g0 + i * V, ww);
      grads(i, yy, zz, dd, ww, pw);
      if (a.dw) part_add<V>(a.dw + wk.wk * a.dim + g0 + i * V, pw, q == 0);
    }
  }
  if (wk.wk >= a.rows || !a.dw) return;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int64_t i = (int64_t)k * wk.tpr + wk.t;
    if (i < np) store_vec<float, V>(a.dw + wk.wk * a.dim + g0 + i * V, dw[k]);
  }
}

// out[c] = sum over parts of part[p][c], in a fixed order: 64 threads per
// column take every 64th part, then their sums are added.  blockIdx.y picks
// one of two (parts, out) pairs.  16 columns per workgroup (64 contiguous
// bytes of each part): enough workgroups for the few thousand columns there
// are (64 columns with 16 threads each took 27 us for 1024 parts of 2 x 2560).
__global__ __launch_bounds__(1024) void s6_norm_colsum(const float* p0, float* o0, const float* p1, float* o1,
                                                       int64_t parts, int64_t dim) {
  __shared__ float buf[64][17];
  const float* p = blockIdx.y ? p1 : p0;
  float* o = blockIdx.y ? o1 : o0;
  if (!o) return;
  const int l = threadIdx.x & 15, r = threadIdx.x >> 4;
  const int64_t c = (int64_t)blockIdx.x * 16 + l;
  float s = 0.0f;
  if (c < dim) {
#pragma unroll 4
    for (int64_t i = r; i < parts; i += 64) s += p[i * dim + c];
  }
  buf[r][l] = s;
  __syncthreads();
  if (threadIdx.x < 256) {  // 16 threads per column
    const int cc = threadIdx.x >> 4, k = threadIdx.x & 15;
    s = (buf[k][cc] + buf[k + 16][cc]) + (buf[k + 32][cc] + buf[k + 48][cc]);
    s = row_sum(s);
    const int64_t co = (int64_t)blockIdx.x * 16 + cc;
    if (k == 0 && co < dim) o[co] = s;
  }
}

// How rows of `width` values are shared out: the pieces' size and number per
// thread, threads of a workgroup, rows per workgroup.
struct NormPlan {
  bool vec, multi, wide;  // wide: a row does not fit the registers
  int K, threads, per;
  int64_t blocks;
};
// A wave per row up to 512 values (256 without 16-byte accesses); above, one
// piece per thread (four single values without 16-byte accesses) up to 1024
// threads; wider rows take 512 threads of two pieces and read the rest again.
// More threads with fewer values each leave room for more waves: with 256
// threads of up to four pieces, the training pass of 16384 rows of 2560 took
// 383 us (200 VGPRs and more, 1 or 2 waves per SIMD).
NormPlan norm_plan(int64_t rows, int64_t width, bool vec, bool sums) {
  NormPlan p;
  p.vec = vec;
  const int64_t np = vec ? width / 8 : width;
  p.K = vec ? (np <= kMaxT ? 1 : 2) : 4;
  p.multi = np <= 64 * p.K;
  const int64_t most_t = p.K == 2 ? 512 : kMaxT;
  int64_t t = (np + p.K - 1) / p.K;
  t = (t + 63) / 64 * 64;
  p.threads = p.multi ? 256 : (int)(t < most_t ? t : most_t);
  p.per = p.multi ? 4 : 1;
  p.wide = !p.multi && np > (int64_t)p.K * p.threads;
  const int64_t need = (rows + p.per - 1) / p.per;
  // Enough workgroups for 2048 threads per CU, where column sums are taken at most
  // kParts walkers.  The forward kernels are resident so; the backward kernels'
  // 104 to 128 VGPRs hold 1024 threads per CU: bf16 rows of 5120 are ten waves, of
  // which one workgroup fits, rows of 2560 five, of which three fit (1024 walkers
  // are then a round and a third).
  int64_t most = (int64_t)cu_count() * (2048 / p.threads);
  if (sums && most > kParts / p.per) most = kParts / p.per;
  p.blocks = need < most ? need : most;
  return p;
}

#define S6_LAUNCH_NORM(kernel, ...)                                                                            \
  do {                                                                                                         \
    const dim3 block((unsigned)p.threads);                                                                     \
    if (!p.vec) {                                                                                              \
      if (p.multi) hipLaunchKernelGGL((kernel<__VA_ARGS__, 1, 4, true, false>), grid, block, 0, st, a);        \
      else if (!p.wide) hipLaunchKernelGGL((kernel<__VA_ARGS__, 1, 4, false, false>), grid, block, 0, st, a);  \
      else hipLaunchKernelGGL((kernel<__VA_ARGS__, 1, 4, false, true>), grid, block, 0, st, a);                \
    } else if (p.multi) hipLaunchKernelGGL((kernel<__VA_ARGS__, 8, 1, true, false>), grid, block, 0, st, a);   \
    else if (p.K == 1) hipLaunchKernelGGL((kernel<__VA_ARGS__, 8, 1, false, false>), grid, block, 0, st, a);   \
    else hipLaunchKernelGGL((kernel<__VA_ARGS__, 8, 2, false, true>), grid, block, 0, st, a);                  \
    S6_HIP(hipGetLastError(), #kernel " launch");                                                              \
  } while (0)

int launch_colsum(const float* p0, float* o0, const float* p1, float* o1, int64_t parts, int64_t dim, hipStream_t st) {
  hipLaunchKernelGGL(s6_norm_colsum, dim3((unsigned)((dim + 15) / 16), 2), dim3(1024), 0, st, p0, o0, p1, o1, parts,
                     dim);
  S6_HIP(hipGetLastError(), "s6_norm_colsum launch");
  return S6_OK;
}

int check_norm(int64_t rows, int64_t dim, int64_t groups, int in_dtype, int64_t s1, int64_t s2) {
  if (in_dtype != S6_F32 && in_dtype != S6_BF16) return S6_ERR_DTYPE;
  if (rows < 0 || dim < 1 || groups < 1 || groups > 65535 || dim % groups) return S6_ERR_SHAPE;
  int64_t t;
  if (!mul_ok(rows, dim, &t) || !mul_ok(t, 8, &t) || dim > INT32_MAX) return S6_ERR_SHAPE;
  const int64_t st[] = {s1, s2};
  for (int64_t s : st)
    if ((rows > 1 && s < dim) || s < 0 || !mul_ok(rows, s, &t) || !mul_ok(t, 8, &t)) return S6_ERR_SHAPE;
  return S6_OK;
}

// Rows start on 16-byte boundaries.
bool row_vec(const void* p, int64_t stride, size_t esz) { return aligned(p, 16) && (stride * (int64_t)esz) % 16 == 0; }

// Room for the parts of one column sum.
size_t part_bytes(int64_t rows, int64_t dim) {
  return up256((size_t)(rows < kParts ? rows : kParts) * (size_t)dim * sizeof(float));
}

}  // namespace

}  // namespace s6i

using namespace s6i;

extern "C" {

int s6_add_norm_fwd(int64_t rows, int64_t dim, int in_dtype, int res_dtype, const void* x, int64_t x_stride,
                    const void* residual, const float* weight, const float* gamma, float scale, float eps, void* out,
                    void* residual_out, void* stream) {
  const int rc = check_norm(rows, dim, 1, in_dtype, x_stride, dim);
  if (rc) return rc;
  if (res_dtype != S6_F32 && res_dtype != in_dtype) return S6_ERR_DTYPE;
  if (rows == 0) return S6_OK;
  if (!x || !weight || !out || !residual_out) return S6_ERR_NULL;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4, rsz = res_dtype == S6_BF16 ? 2 : 4;
  if (!aligned(x, esz) || !aligned(out, esz) || !aligned(residual, rsz) || !aligned(residual_out, rsz) ||
      !aligned(weight, 4) || !aligned(gamma, 4))
    return S6_ERR_ALIGN;
  const bool vec = dim % 8 == 0 && row_vec(x, x_stride, esz) && aligned(out, 16) && aligned(residual, 16) &&
                   aligned(residual_out, 16) && aligned(weight, 16) && aligned(gamma, 16);
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.rows = rows; a.dim = dim; a.gd = dim; a.a = x; a.a_stride = x_stride; a.b = residual; a.w = weight; a.gamma = gamma;
  a.scale = scale; a.eps = eps; a.o1 = out; a.o2 = residual_out;
  const NormPlan p = norm_plan(rows, dim, vec, false);
  const dim3 grid((unsigned)p.blocks);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_kernel, float, float);
  else if (res_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_kernel, uint16_t, float);
  else S6_LAUNCH_NORM(s6_add_norm_kernel, uint16_t, uint16_t);
  return S6_OK;
}

int s6_add_norm_q8_fwd(int64_t rows, int64_t dim, int in_dtype, int res_dtype, const void* x, int64_t x_stride,
                       const void* residual, const float* weight, const float* gamma, float scale, float eps, void* out,
                       float* out_scale, void* residual_out, void* stream) {
  const int rc = check_norm(rows, dim, 1, in_dtype, x_stride, dim);
  if (rc) return rc;
  if (res_dtype != S6_F32 && res_dtype != in_dtype) return S6_ERR_DTYPE;
  if (rows == 0) return S6_OK;
  if (!x || !weight || !out || !out_scale || !residual_out) return S6_ERR_NULL;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4, rsz = res_dtype == S6_BF16 ? 2 : 4;
  if (!aligned(x, esz) || !aligned(out_scale, 4) || !aligned(residual, rsz) || !aligned(residual_out, rsz) ||
      !aligned(weight, 4) || !aligned(gamma, 4))
    return S6_ERR_ALIGN;
  const bool vec = dim % 8 == 0 && row_vec(x, x_stride, esz) && aligned(out, 8) && aligned(residual, 16) &&
                   aligned(residual_out, 16) && aligned(weight, 16) && aligned(gamma, 16);
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.rows = rows; a.dim = dim; a.gd = dim; a.a = x; a.a_stride = x_stride; a.b = residual; a.w = weight; a.gamma = gamma;
  a.scale = scale; a.eps = eps; a.o1 = out; a.o2 = residual_out; a.row_scale = out_scale;
  const NormPlan p = norm_plan(rows, dim, vec, false);
  const dim3 grid((unsigned)p.blocks);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_q8_kernel, float, float);
  else if (res_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_q8_kernel, uint16_t, float);
  else S6_LAUNCH_NORM(s6_add_norm_q8_kernel, uint16_t, uint16_t);
  return S6_OK;
}

int s6_add_norm_bwd_workspace_size(int64_t rows, int64_t dim, size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  const int rc = check_norm(rows, dim, 1, S6_F32, dim, dim);
  if (rc) return rc;
  *bytes = rows ? 2 * part_bytes(rows, dim) : 0;
  return S6_OK;
}

int s6_add_norm_bwd(int64_t rows, int64_t dim, int in_dtype, int res_dtype, const void* dout,
                    const void* dresidual_out, const void* residual_out, const void* x, int64_t x_stride,
                    const float* weight, const float* gamma, float scale, float eps, void* dx, void* dresidual,
                    float* dweight, float* dgamma, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_norm(rows, dim, 1, in_dtype, x ? x_stride : dim, dim);
  if (rc) return rc;
  if (res_dtype != S6_F32 && res_dtype != in_dtype) return S6_ERR_DTYPE;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (rows == 0) {  // empty sums
    fill(dweight, 0.0f, dim, st);
    fill(dgamma, 0.0f, dim, st);
    S6_HIP(hipGetLastError(), "fill launch");
    return S6_OK;
  }
  if (!dout || !residual_out || !weight || (!dx && !dresidual && !dweight)) return S6_ERR_NULL;
  if (gamma ? (!dgamma || !x) : dgamma != nullptr) return S6_ERR_NULL;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4, rsz = res_dtype == S6_BF16 ? 2 : 4;
  if (!aligned(dout, esz) || !aligned(x, esz) || !aligned(dx, esz) || !aligned(dresidual_out, rsz) ||
      !aligned(residual_out, rsz) || !aligned(dresidual, rsz) || !aligned(weight, 4) || !aligned(gamma, 4) ||
      !aligned(dweight, 4) || !aligned(dgamma, 4))
    return S6_ERR_ALIGN;
  const size_t part = part_bytes(rows, dim);
  const bool sums = dweight || dgamma;
  if (sums) {
    if (!workspace || workspace_bytes < 2 * part) return S6_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return S6_ERR_ALIGN;
  }
  const bool vec = dim % 8 == 0 && aligned(dout, 16) && (!dgamma || row_vec(x, x_stride, esz)) && aligned(dx, 16) &&
                   aligned(dresidual_out, 16) && aligned(residual_out, 16) && aligned(dresidual, 16) &&
                   aligned(weight, 16) && aligned(gamma, 16);
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.rows = rows; a.dim = dim; a.gd = dim; a.a = x; a.a_stride = x_stride; a.dout = dout; a.dres = dresidual_out;
  a.res = residual_out; a.w = weight; a.gamma = gamma; a.scale = scale; a.eps = eps; a.o1 = dx; a.o2 = dresidual;
  a.dw = dweight ? static_cast<float*>(workspace) : nullptr;
  a.dg = dgamma ? reinterpret_cast<float*>(static_cast<char*>(workspace) + part) : nullptr;
  const NormPlan p = norm_plan(rows, dim, vec, sums);
  const dim3 grid((unsigned)p.blocks);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_bwd_kernel, float, float);
  else if (res_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_bwd_kernel, uint16_t, float);
  else S6_LAUNCH_NORM(s6_add_norm_bwd_kernel, uint16_t, uint16_t);
  if (!sums) return S6_OK;
  const int64_t walkers = p.blocks * p.per, parts = walkers < rows ? walkers : rows;
  return launch_colsum(a.dw, dweight, a.dg, dgamma, parts, dim, st);
}

int s6_gated_norm_fwd(int64_t rows, int64_t dim, int64_t groups, int in_dtype, int flags, const void* y,
                      int64_t y_stride, const void* z, int64_t z_stride, const float* weight, float eps, void* out,
                      void* stream) {
  const int rc = check_norm(rows, dim, groups, in_dtype, y_stride, z ? z_stride : dim);
  if (rc) return rc;
  if (flags & ~S6_GATE_AFTER) return S6_ERR_FLAGS;
  if (rows == 0) return S6_OK;
  if (!y || !weight || !out) return S6_ERR_NULL;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4;
  if (!aligned(y, esz) || !aligned(z, esz) || !aligned(out, esz) || !aligned(weight, 4)) return S6_ERR_ALIGN;
  const bool vec = (dim / groups) % 8 == 0 && row_vec(y, y_stride, esz) && (!z || row_vec(z, z_stride, esz)) &&
                   aligned(out, 16) && aligned(weight, 16);
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.rows = rows; a.dim = dim; a.gd = dim / groups; a.a = y; a.a_stride = y_stride; a.b = z; a.b_stride = z_stride;
  a.w = weight; a.eps = eps; a.after = (flags & S6_GATE_AFTER) != 0; a.o1 = out;
  const NormPlan p = norm_plan(rows, a.gd, vec, false);
  const dim3 grid((unsigned)p.blocks, (unsigned)groups);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_gated_norm_kernel, float);
  else S6_LAUNCH_NORM(s6_gated_norm_kernel, uint16_t);
  return S6_OK;
}

int s6_gated_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t groups, size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  const int rc = check_norm(rows, dim, groups, S6_F32, dim, dim);
  if (rc) return rc;
  *bytes = rows ? part_bytes(rows, dim) : 0;
  return S6_OK;
}

int s6_gated_norm_bwd(int64_t rows, int64_t dim, int64_t groups, int in_dtype, int flags, const void* dout,
                      const void* y, int64_t y_stride, const void* z, int64_t z_stride, const float* weight, float eps,
                      void* dy, void* dz, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_norm(rows, dim, groups, in_dtype, y_stride, z ? z_stride : dim);
  if (rc) return rc;
  if (flags & ~S6_GATE_AFTER) return S6_ERR_FLAGS;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (rows == 0) {
    fill(dweight, 0.0f, dim, st);
    S6_HIP(hipGetLastError(), "fill launch");
    return S6_OK;
  }
  if (!dout || !y || !weight || !dy || (z && !dz)) return S6_ERR_NULL;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4;
  if (!aligned(dout, esz) || !aligned(y, esz) || !aligned(z, esz) || !aligned(dy, esz) || !aligned(dz, esz) ||
      !aligned(weight, 4) || !aligned(dweight, 4))
    return S6_ERR_ALIGN;
  if (dweight) {
    if (!workspace || workspace_bytes < part_bytes(rows, dim)) return S6_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return S6_ERR_ALIGN;
  }
  const bool vec = (dim / groups) % 8 == 0 && aligned(dout, 16) && row_vec(y, y_stride, esz) &&
                   (!z || (row_vec(z, z_stride, esz) && aligned(dz, 16))) && aligned(dy, 16) && aligned(weight, 16);
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.rows = rows; a.dim = dim; a.gd = dim / groups; a.a = y; a.a_stride = y_stride; a.b = z; a.b_stride = z_stride;
  a.dout = dout; a.w = weight; a.eps = eps; a.after = (flags & S6_GATE_AFTER) != 0; a.o1 = dy; a.o2 = dz;
  a.dw = dweight ? static_cast<float*>(workspace) : nullptr;
  const NormPlan p = norm_plan(rows, a.gd, vec, dweight != nullptr);
  const dim3 grid((unsigned)p.blocks, (unsigned)groups);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_gated_norm_bwd_kernel, float);
  else S6_LAUNCH_NORM(s6_gated_norm_bwd_kernel, uint16_t);
  if (!dweight) return S6_OK;
  const int64_t walkers = p.blocks * p.per, parts = walkers < rows ? walkers : rows;
  return launch_colsum(a.dw, dweight, nullptr, nullptr, parts, dim, st);
}

}  // extern "C"
