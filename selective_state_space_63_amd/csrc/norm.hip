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
// the row's threads once and writes its outputs: the kernels are bound by
// HBM.  Sums and statistics are fp32.
//
// Layout: TPR threads (a wave, or a workgroup of four) per row, K pieces of V
// consecutive values per thread in registers (V = 8: 16-byte accesses; V = 1
// where a width, stride or pointer does not allow them); rows wider than K V
// TPR read the rest again in the second phase.  A thread keeps its columns
// over the rows it walks, so weights are read once per thread and the column
// sums (dw, dgamma) stay in registers until the end; their per-thread-group
// parts are then added in a fixed order by s6_norm_colsum.
#include "block_internal.h"

namespace s6i {

namespace {

constexpr int kK = 4;  // register pieces per thread

// Most row walkers where column sums are taken (a walker leaves one part of
// them): 512 workgroups either way, of four waves with a row each for rows
// that a wave holds, of four waves on one row for wider ones.
int64_t most_parts(int64_t width, int tpr) { return width <= (int64_t)kK * 64 * 8 && tpr == 64 ? 2048 : 512; }

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
};

// Sum of two values over the TPR threads of a row.  For TPR = 256 the four
// waves meet in LDS; the buffer alternates between two halves, so one barrier
// per row is enough (a wave writes half i again only after the barrier of
// half i + 1, which every wave reaches after reading half i).
template <int TPR>
__device__ __forceinline__ void row_sum2(float& s, float& t, float (*buf)[2][4], int par) {
  s = wave_sum(s);
  t = wave_sum(t);
  if constexpr (TPR > 64) {
    const int w = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) { buf[par][0][w] = s; buf[par][1][w] = t; }
    __syncthreads();
    s = (buf[par][0][0] + buf[par][0][1]) + (buf[par][0][2] + buf[par][0][3]);
    t = (buf[par][1][0] + buf[par][1][1]) + (buf[par][1][2] + buf[par][1][3]);
  }
}

__device__ __forceinline__ float sigmoid_f(float z) { return fast_rcp(1.0f + fast_exp2(-z * kLog2e)); }

// Walker `wk` of `nw` takes rows wk, wk + nw, ...: every walker of a
// workgroup makes the same number of turns (barriers), masked past the end.
struct Walk {
  int64_t wk, nw, turns;
  int t;
};
template <int TPR>
__device__ __forceinline__ Walk walk_of(int64_t rows) {
  Walk o;
  constexpr int per = 256 / TPR;
  o.nw = (int64_t)gridDim.x * per;
  o.wk = (int64_t)blockIdx.x * per + threadIdx.x / TPR;
  o.turns = (rows + o.nw - 1) / o.nw;
  o.t = threadIdx.x % TPR;
  return o;
}

// ------------------------------------------------------------- add norm --
template <typename In, typename Res, int V, int TPR>
__global__ __launch_bounds__(256) void s6_add_norm_kernel(NormArgs a) {
  __shared__ float buf[2][2][4];
  const Walk wk = walk_of<TPR>(a.rows);
  const int64_t np = (a.dim + V - 1) / V;  // pieces of a row
  const float inv_d = 1.0f / (float)a.dim;
  float w[kK][V], ga[kK][V];
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int64_t i = (int64_t)k * TPR + wk.t;
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
  for (int64_t q = 0; q < wk.turns; ++q) {
    const int64_t row = q * wk.nw + wk.wk;
    const bool on = row < a.rows;
    const In* x = static_cast<const In*>(a.a) + row * a.a_stride;
    const Res* r = a.b ? static_cast<const Res*>(a.b) + row * a.dim : nullptr;
    In* out = static_cast<In*>(a.o1) + row * a.dim;
    Res* ro = static_cast<Res*>(a.o2) + row * a.dim;
    float u[kK][V], rv[kK][V];
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
        load_vec<In, V>(x + i * V, u[k]);
        if (r) load_vec<Res, V>(r + i * V, rv[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
#pragma unroll
        for (int j = 0; j < V; ++j) {
          u[k][j] = r ? __builtin_fmaf(ga[k][j], u[k][j], rv[k][j]) : ga[k][j] * u[k][j];
          s = __builtin_fmaf(u[k][j], u[k][j], s);
        }
        store_vec<Res, V>(ro + i * V, u[k]);
      }
    }
    // the sum of a piece past the registers: r' is formed again for out, from
    // x and the residual, so it is stored in the second phase (residual_out
    // may be the residual's buffer)
    auto wide = [&](int64_t i, float (&v)[V]) {
      float rr[V], gg[V];
      load_vec<In, V>(x + i * V, v);
      if (r) load_vec<Res, V>(r + i * V, rr);
      if (a.gamma) load_vec<float, V>(a.gamma + i * V, gg);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float g = a.gamma ? gg[j] * a.scale : a.scale;
        v[j] = r ? __builtin_fmaf(g, v[j], rr[j]) : g * v[j];
      }
    };
    for (int64_t i = (int64_t)kK * TPR + wk.t; on && i < np; i += TPR) {
      float v[V];
      wide(i, v);
#pragma unroll
      for (int j = 0; j < V; ++j) s = __builtin_fmaf(v[j], v[j], s);
    }
    row_sum2<TPR>(s, unused, buf, (int)(q & 1));
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_d, a.eps));
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
#pragma unroll
        for (int j = 0; j < V; ++j) u[k][j] = u[k][j] * inv * w[k][j];
        store_vec<In, V>(out + i * V, u[k]);
      }
    }
    for (int64_t i = (int64_t)kK * TPR + wk.t; on && i < np; i += TPR) {
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

template <typename In, typename Res, int V, int TPR>
__global__ __launch_bounds__(256) void s6_add_norm_bwd_kernel(NormArgs a) {
  __shared__ float buf[2][2][4];
  const Walk wk = walk_of<TPR>(a.rows);
  const int64_t np = (a.dim + V - 1) / V;
  const float inv_d = 1.0f / (float)a.dim;
  float w[kK][V], ga[kK][V], dw[kK][V], dg[kK][V];
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int64_t i = (int64_t)k * TPR + wk.t;
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
    float u[kK][V], d[kK][V], e[kK][V];
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
        load_vec<Res, V>(res + i * V, u[k]);
        load_vec<In, V>(dout + i * V, d[k]);
        if (dres) load_vec<Res, V>(dres + i * V, e[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          s = __builtin_fmaf(u[k][j], u[k][j], s);
          t = __builtin_fmaf(d[k][j] * w[k][j], u[k][j], t);
        }
    }
    for (int64_t i = (int64_t)kK * TPR + wk.t; on && i < np; i += TPR) {
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
    row_sum2<TPR>(s, t, buf, (int)(q & 1));
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_d, a.eps));
    const float m = inv * inv * (t * inv_d);  // u i m = u m, with m including both factors i
    auto grads = [&](int64_t i, const float (&uu)[V], const float (&dd)[V], const float (&ee)[V], const float (&ww)[V],
                     const float (&gg)[V], float (&pw)[V], float (&pg)[V]) {
      float o[V], xv[V];
      if (a.dg) load_vec<In, V>(x + i * V, xv);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        pw[j] = dd[j] * (uu[j] * inv);
        o[j] = inv * __builtin_fmaf(-uu[j], m, dd[j] * ww[j]) + (dres ? ee[j] : 0.0f);
      }
      if (dr) store_vec<Res, V>(dr + i * V, o);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        pg[j] = a.dg ? a.scale * (o[j] * xv[j]) : 0.0f;
        o[j] *= gg[j];
      }
      if (dx) store_vec<In, V>(dx + i * V, o);
    };
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
        float pw[V], pg[V];
        grads(i, u[k], d[k], e[k], w[k], ga[k], pw, pg);
#pragma unroll
        for (int j = 0; j < V; ++j) { dw[k][j] += pw[j]; dg[k][j] += pg[j]; }
      }
    }
    for (int64_t i = (int64_t)kK * TPR + wk.t; on && i < np; i += TPR) {
      float uu[V], dd[V], ee[V], ww[V], gg[V], pw[V], pg[V];
      load_vec<Res, V>(res + i * V, uu);
      load_vec<In, V>(dout + i * V, dd);
      if (dres) load_vec<Res, V>(dres + i * V, ee);
      load_vec<float, V>(a.w + i * V, ww);
      if (a.gamma) load_vec<float, V>(a.gamma + i * V, gg);
#pragma unroll
      for (int j = 0; j < V; ++j) gg[j] = a.gamma ? gg[j] * a.scale : a.scale;
      grads(i, uu, dd, ee, ww, gg, pw, pg);
      if (a.dw) part_add<V>(a.dw + wk.wk * a.dim + i * V, pw, q == 0);
      if (a.dg) part_add<V>(a.dg + wk.wk * a.dim + i * V, pg, q == 0);
    }
  }
  if (wk.wk >= a.rows) return;  // no row of its own: its part is not read
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int64_t i = (int64_t)k * TPR + wk.t;
    if (i < np) {
      if (a.dw) store_vec<float, V>(a.dw + wk.wk * a.dim + i * V, dw[k]);
      if (a.dg) store_vec<float, V>(a.dg + wk.wk * a.dim + i * V, dg[k]);
    }
  }
}

// ----------------------------------------------------------- gated norm --
// blockIdx.y: the group.
template <typename In, int V, int TPR>
__global__ __launch_bounds__(256) void s6_gated_norm_kernel(NormArgs a) {
  __shared__ float buf[2][2][4];
  const Walk wk = walk_of<TPR>(a.rows);
  const int64_t np = (a.gd + V - 1) / V, g0 = (int64_t)blockIdx.y * a.gd;
  const float inv_d = 1.0f / (float)a.gd;
  float w[kK][V];
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int64_t i = (int64_t)k * TPR + wk.t;
    if (i < np) load_vec<float, V>(a.w + g0 + i * V, w[k]);
  }
  for (int64_t q = 0; q < wk.turns; ++q) {
    const int64_t row = q * wk.nw + wk.wk;
    const bool on = row < a.rows;
    const In* y = static_cast<const In*>(a.a) + row * a.a_stride + g0;
    const In* z = a.b ? static_cast<const In*>(a.b) + row * a.b_stride + g0 : nullptr;
    In* out = static_cast<In*>(a.o1) + row * a.dim + g0;
    float u[kK][V], zv[kK][V];
    float s = 0.0f, unused = 0.0f;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
        load_vec<In, V>(y + i * V, u[k]);
        if (z) load_vec<In, V>(z + i * V, zv[k]);
      }
    }
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
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
        gate(u[k], zv[k]);
#pragma unroll
        for (int j = 0; j < V; ++j) s = __builtin_fmaf(u[k][j], u[k][j], s);
      }
    }
    for (int64_t i = (int64_t)kK * TPR + wk.t; on && i < np; i += TPR) {
      float v[V], f[V];
      load_vec<In, V>(y + i * V, v);
      if (z) load_vec<In, V>(z + i * V, f);
      gate(v, f);
#pragma unroll
      for (int j = 0; j < V; ++j) s = __builtin_fmaf(v[j], v[j], s);
    }
    row_sum2<TPR>(s, unused, buf, (int)(q & 1));
    const float inv = __builtin_amdgcn_rsqf(__builtin_fmaf(s, inv_d, a.eps));
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
#pragma unroll
        for (int j = 0; j < V; ++j) u[k][j] = u[k][j] * inv * w[k][j] * zv[k][j];
        store_vec<In, V>(out + i * V, u[k]);
      }
    }
    for (int64_t i = (int64_t)kK * TPR + wk.t; on && i < np; i += TPR) {
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

template <typename In, int V, int TPR>
__global__ __launch_bounds__(256) void s6_gated_norm_bwd_kernel(NormArgs a) {
  __shared__ float buf[2][2][4];
  const Walk wk = walk_of<TPR>(a.rows);
  const int64_t np = (a.gd + V - 1) / V, g0 = (int64_t)blockIdx.y * a.gd;
  const float inv_d = 1.0f / (float)a.gd;
  float w[kK][V], dw[kK][V];
#pragma unroll
  for (int k = 0; k < kK; ++k) {
    const int64_t i = (int64_t)k * TPR + wk.t;
#pragma unroll
    for (int j = 0; j < V; ++j) dw[k][j] = 0.0f;
    if (i < np) load_vec<float, V>(a.w + g0 + i * V, w[k]);
  }
  for (int64_t q = 0; q < wk.turns; ++q) {
    const int64_t row = q * wk.nw + wk.wk;
    const bool on = row < a.rows;
    const In* y = static_cast<const In*>(a.a) + row * a.a_stride + g0;
    const In* z = a.b ? static_cast<const In*>(a.b) + row * a.b_stride + g0 : nullptr;
    const In* dout = static_cast<const In*>(a.dout) + row * a.dim + g0;
    In* dy = static_cast<In*>(a.o1) + row * a.dim + g0;
    In* dz = z ? static_cast<In*>(a.o2) + row * a.dim + g0 : nullptr;
    float yv[kK][V], zv[kK][V], d[kK][V];
    float s = 0.0f, t = 0.0f;
#pragma unroll
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
        load_vec<In, V>(y + i * V, yv[k]);
        load_vec<In, V>(dout + i * V, d[k]);
        if (z) load_vec<In, V>(z + i * V, zv[k]);
      }
    }
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
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) sums(yv[k], zv[k], d[k], w[k]);
    }
    for (int64_t i = (int64_t)kK * TPR + wk.t; on && i < np; i += TPR) {
      float yy[V], zz[V], dd[V], ww[V];
      load_vec<In, V>(y + i * V, yy);
      load_vec<In, V>(dout + i * V, dd);
      if (z) load_vec<In, V>(z + i * V, zz);
      load_vec<float, V>(a.w + g0 + i * V, ww);
      sums(yy, zz, dd, ww);
    }
    row_sum2<TPR>(s, t, buf, (int)(q & 1));
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
    for (int k = 0; k < kK; ++k) {
      const int64_t i = (int64_t)k * TPR + wk.t;
      if (on && i < np) {
        float pw[V];
        grads(i, yv[k], zv[k], d[k], w[k], pw);
#pragma unroll
        for (int j = 0; j < V; ++j) dw[k][j] += pw[j];
      }
    }
    for (int64_t i = (int64_t)kK * TPR + wk.t; on && i < np; i += TPR) {
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
  for (int k = 0; k < kK; ++k) {
    const int64_t i = (int64_t)k * TPR + wk.t;
    if (i < np) store_vec<float, V>(a.dw + wk.wk * a.dim + g0 + i * V, dw[k]);
  }
}

// out[c] = sum over parts of part[p][c], in a fixed order: 16 threads per
// column take every 16th part, then their sums are added.  blockIdx.y picks
// one of two (parts, out) pairs.
__global__ __launch_bounds__(1024) void s6_norm_colsum(const float* p0, float* o0, const float* p1, float* o1,
                                                       int64_t parts, int64_t dim) {
  __shared__ float buf[16][64];
  const float* p = blockIdx.y ? p1 : p0;
  float* o = blockIdx.y ? o1 : o0;
  if (!o) return;
  const int l = threadIdx.x & 63, r = threadIdx.x >> 6;
  const int64_t c = (int64_t)blockIdx.x * 64 + l;
  float s = 0.0f;
  if (c < dim)
    for (int64_t i = r; i < parts; i += 16) s += p[i * dim + c];
  buf[r][l] = s;
  __syncthreads();
  if (r == 0 && c < dim) {
    s = buf[0][l];
    for (int i = 1; i < 16; ++i) s += buf[i][l];
    o[c] = s;
  }
}

// Threads per row: a wave where its registers hold the row (512 values with
// 16-byte pieces per register piece), else a workgroup.
int tpr_of(int64_t width, bool vec) { return width <= (int64_t)kK * 64 * (vec ? 8 : 1) ? 64 : 256; }

// Workgroups along the rows: at most most_parts walkers where column sums are
// taken, else enough for every CU to hold eight.
int64_t walk_blocks(int64_t rows, int64_t width, int tpr, bool sums) {
  const int64_t per = 256 / tpr;
  const int64_t need = (rows + per - 1) / per;
  const int64_t most = sums ? most_parts(width, tpr) / per : (int64_t)cu_count() * 8;
  return need < most ? need : most;
}

#define S6_LAUNCH_NORM(kernel, ...)                                                                              \
  do {                                                                                                           \
    if (vec && tpr == 64) hipLaunchKernelGGL((kernel<__VA_ARGS__, 8, 64>), grid, dim3(256), 0, st, a);           \
    else if (vec) hipLaunchKernelGGL((kernel<__VA_ARGS__, 8, 256>), grid, dim3(256), 0, st, a);                  \
    else if (tpr == 64) hipLaunchKernelGGL((kernel<__VA_ARGS__, 1, 64>), grid, dim3(256), 0, st, a);             \
    else hipLaunchKernelGGL((kernel<__VA_ARGS__, 1, 256>), grid, dim3(256), 0, st, a);                           \
    S6_HIP(hipGetLastError(), #kernel " launch");                                                                \
  } while (0)

int launch_colsum(const float* p0, float* o0, const float* p1, float* o1, int64_t parts, int64_t dim, hipStream_t st) {
  hipLaunchKernelGGL(s6_norm_colsum, dim3((unsigned)((dim + 63) / 64), 2), dim3(1024), 0, st, p0, o0, p1, o1, parts,
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

// Room for the parts of one column sum over groups of `width` columns.
size_t part_bytes(int64_t rows, int64_t dim, int64_t width) {
  const int64_t most = most_parts(width, 64);
  return up256((size_t)(rows < most ? rows : most) * (size_t)dim * sizeof(float));
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
  const int tpr = tpr_of(dim, vec);
  const dim3 grid((unsigned)walk_blocks(rows, dim, tpr, false));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_kernel, float, float);
  else if (res_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_kernel, uint16_t, float);
  else S6_LAUNCH_NORM(s6_add_norm_kernel, uint16_t, uint16_t);
  return S6_OK;
}

int s6_add_norm_bwd_workspace_size(int64_t rows, int64_t dim, size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  const int rc = check_norm(rows, dim, 1, S6_F32, dim, dim);
  if (rc) return rc;
  *bytes = rows ? 2 * part_bytes(rows, dim, dim) : 0;
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
  const size_t part = part_bytes(rows, dim, dim);
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
  const int tpr = tpr_of(dim, vec);
  const int64_t blocks = walk_blocks(rows, dim, tpr, sums);
  const dim3 grid((unsigned)blocks);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_bwd_kernel, float, float);
  else if (res_dtype == S6_F32) S6_LAUNCH_NORM(s6_add_norm_bwd_kernel, uint16_t, float);
  else S6_LAUNCH_NORM(s6_add_norm_bwd_kernel, uint16_t, uint16_t);
  if (!sums) return S6_OK;
  const int64_t walkers = blocks * (256 / tpr), parts = walkers < rows ? walkers : rows;
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
  const int tpr = tpr_of(a.gd, vec);
  const dim3 grid((unsigned)walk_blocks(rows, dim, tpr, false), (unsigned)groups);
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_gated_norm_kernel, float);
  else S6_LAUNCH_NORM(s6_gated_norm_kernel, uint16_t);
  return S6_OK;
}

int s6_gated_norm_bwd_workspace_size(int64_t rows, int64_t dim, int64_t groups, size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  const int rc = check_norm(rows, dim, groups, S6_F32, dim, dim);
  if (rc) return rc;
  *bytes = rows ? part_bytes(rows, dim, dim / groups) : 0;
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
    if (!workspace || workspace_bytes < part_bytes(rows, dim, dim / groups)) return S6_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return S6_ERR_ALIGN;
  }
  const bool vec = (dim / groups) % 8 == 0 && aligned(dout, 16) && row_vec(y, y_stride, esz) &&
                   (!z || (row_vec(z, z_stride, esz) && aligned(dz, 16))) && aligned(dy, 16) && aligned(weight, 16);
  NormArgs a;
  memset(&a, 0, sizeof(a));
  a.rows = rows; a.dim = dim; a.gd = dim / groups; a.a = y; a.a_stride = y_stride; a.b = z; a.b_stride = z_stride;
  a.dout = dout; a.w = weight; a.eps = eps; a.after = (flags & S6_GATE_AFTER) != 0; a.o1 = dy; a.o2 = dz;
  a.dw = dweight ? static_cast<float*>(workspace) : nullptr;
  const int tpr = tpr_of(a.gd, vec);
  const int64_t blocks = walk_blocks(rows, a.gd, tpr, dweight != nullptr);
  const dim3 grid((unsigned)blocks, (unsigned)groups);
  if (in_dtype == S6_F32) S6_LAUNCH_NORM(s6_gated_norm_bwd_kernel, float);
  else S6_LAUNCH_NORM(s6_gated_norm_bwd_kernel, uint16_t);
  if (!dweight) return S6_OK;
  const int64_t walkers = blocks * (256 / tpr), parts = walkers < rows ? walkers : rows;
  return launch_colsum(a.dw, dweight, nullptr, nullptr, parts, dim, st);
}

}  // extern "C"
