// heads_step.hip -- the single-token step of the multi-head scan
// (s6_heads_state_update) and the argument checks of the heads entry points.
//
//   S <- e^{s A} S + w x B^T,   y = S C + D x        (S: P x N per head)
//
// The state is read and written once: 8 P N bytes per head beside about
// 4 (P + N) of inputs and outputs, so the step is bound by HBM (or by the
// launch, for one sequence).  Layout: LPR adjacent lanes hold a state row of
// N <= 4 LPR values, four consecutive values each (16-byte accesses that are
// contiguous over a wave), and K rows per lane so that K loads are in flight
// before the first is used; B and C are the same for all of a lane's rows
// and stay in registers.  The row's dot product with C is added over its
// lanes with DPP.
//
// 256 sequences of 80 heads of 64, N 128: 248 us, 5.4 TB/s of the 6.2 TB/s
// that a copy reaches (265 us with the inputs loaded behind the state's use);
// one sequence of 24 heads: 4 us of kernel, 12.6 us with the call.
#include "block_internal.h"

namespace s6i {

namespace {

struct StepHeadsArgs {
  float* h;
  const void* x;
  const void* delta;
  const float* dbias;
  const float* A;
  const void* Bm;
  const void* Cm;
  const float* D;
  void* y;
  int softplus, unit;
  int heads, headdim, hpg, dstate;  // hpg: heads per group
  int64_t x_batch, delta_batch, b_batch, c_batch;
};

// Four values p[0..3] of a row of n, 0 past its end.
template <typename In, bool VEC>
__device__ __forceinline__ void load4_in(const In* p, int n, float (&f)[4]) {
  if constexpr (VEC) {
    if (n >= 4) {
      load_vec<In, 4>(p, f);
    } else {
      f[0] = f[1] = f[2] = f[3] = 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < n ? to_f32(p[j]) : 0.0f;
  }
}

// LPR lanes per state row; 256/LPR rows at a time, K times.  blockIdx.x: the
// row block of a head; blockIdx.y, z: (sequence, head).  VEC: dstate is a
// multiple of 4, and h, Bm, Cm rows are aligned to four values.
template <typename In, int LPR, int K, bool VEC>
__global__ __launch_bounds__(256) void s6_heads_step_kernel(StepHeadsArgs a, int64_t pairs) {
  const int64_t pair = (int64_t)blockIdx.z * 65535 + blockIdx.y;
  if (pair >= pairs) return;
  const int64_t b = pair / a.heads;
  const int hd = (int)(pair - b * a.heads);
  const int l = threadIdx.x % LPR, rw = threadIdx.x / LPR;
  constexpr int kRows = 256 / LPR;
  const int p0 = blockIdx.x * (kRows * K) + rw;
  const int n0 = 4 * l, nleft = a.dstate - n0;
  float* hrow = a.h + (pair * a.headdim) * (int64_t)a.dstate + n0;
  float s[K][4];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = p0 + k * kRows;
    const int left = p < a.headdim ? nleft : 0;
    load4_in<float, VEC>(hrow + (int64_t)p * a.dstate, left, s[k]);
  }
  float xv[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = p0 + k * kRows;
    xv[k] = p < a.headdim ? to_f32(static_cast<const In*>(a.x)[b * a.x_batch + (int64_t)hd * a.headdim + p]) : 0.0f;
  }
  float Bv[4], Cv[4];
  const int64_t gof = (int64_t)(hd / a.hpg) * a.dstate + n0;
  load4_in<In, VEC>(static_cast<const In*>(a.Bm) + b * a.b_batch + gof, nleft, Bv);
  load4_in<In, VEC>(static_cast<const In*>(a.Cm) + b * a.c_batch + gof, nleft, Cv);
  float st = 1.0f;
  if (a.delta) {
    st = to_f32(static_cast<const In*>(a.delta)[b * a.delta_batch + hd]) + (a.dbias ? a.dbias[hd] : 0.0f);
    if (a.softplus) st = softplus_f(st);
  }
  const float e = fast_exp2(clamp_log2(st * a.A[hd] * kLog2e));
  const float w = a.unit ? 1.0f : st;
  const float dsk = a.D ? a.D[hd] : 0.0f;
  In* y = static_cast<In*>(a.y) + pair * a.headdim;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int p = p0 + k * kRows;
    const float wx = w * xv[k];
    float dot = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[k][j] = __builtin_fmaf(e, s[k][j], wx * Bv[j]);
      if (j < nleft) dot = __builtin_fmaf(s[k][j], Cv[j], dot);
    }
    if (p < a.headdim) {
      float* hp = hrow + (int64_t)p * a.dstate;
      if constexpr (VEC) {
        if (nleft >= 4) store_vec<float, 4>(hp, s[k]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < nleft) hp[j] = s[k][j];
      }
    }
    // lanes past dstate add nothing (their values could be NaN: 0 times an infinite x)
    dot += dpp_f<0xB1>(dot);
    dot += dpp_f<0x4E>(dot);
    dot += dpp_f<0x141>(dot);
    if constexpr (LPR >= 16) dot += dpp_f<0x140>(dot);
    if constexpr (LPR >= 32) dot = pair_row_sum(dot);
    if (l == 0 && p < a.headdim) y[p] = from_f32<In>(__builtin_fmaf(dsk, xv[k], dot));
  }
}

template <typename In, int LPR, int K>
int launch_step(const StepHeadsArgs& a, int64_t pairs, bool vec, hipStream_t st) {
  constexpr int rows = 256 / LPR * K;
  const dim3 grid((unsigned)((a.headdim + rows - 1) / rows), (unsigned)(pairs < 65535 ? pairs : 65535),
                  (unsigned)((pairs + 65534) / 65535));
  if (vec)
    hipLaunchKernelGGL((s6_heads_step_kernel<In, LPR, K, true>), grid, dim3(256), 0, st, a, pairs);
  else
    hipLaunchKernelGGL((s6_heads_step_kernel<In, LPR, K, false>), grid, dim3(256), 0, st, a, pairs);
  S6_HIP(hipGetLastError(), "s6_heads_step_kernel launch");
  return S6_OK;
}

template <typename In>
int dispatch_step(const StepHeadsArgs& a, int64_t pairs, bool vec, hipStream_t st) {
  if (a.dstate > 64) return launch_step<In, 32, 4>(a, pairs, vec, st);
  if (a.dstate > 32) return launch_step<In, 16, 4>(a, pairs, vec, st);
  return launch_step<In, 8, 2>(a, pairs, vec, st);
}

}  // namespace

int check_heads(const s6_heads_dims* d, int in_dtype, int flags, bool has_delta, bool has_bias, bool tokens) {
  if (!d) return S6_ERR_NULL;
  if (in_dtype != S6_F32 && in_dtype != S6_BF16) return S6_ERR_DTYPE;
  if (flags & ~(S6_DELTA_SOFTPLUS | S6_UNIT_INPUT)) return S6_ERR_FLAGS;
  if (d->batch < 0 || d->heads < 0 || d->headdim < 1 || d->groups < 1 || (tokens && d->seqlen < 0)) return S6_ERR_SHAPE;
  if (d->dstate < 1 || d->dstate > kMaxHeadState) return S6_ERR_UNSUPPORTED;
  if (d->heads % d->groups) return S6_ERR_SHAPE;
  if (d->batch == 0 || d->heads == 0) return S6_OK;
  // a bias or a softplus acts on delta: without one there is nothing to act on
  if (!has_delta && (has_bias || (flags & S6_DELTA_SOFTPLUS)) && !(tokens && d->seqlen == 0)) return S6_ERR_NULL;
  const int64_t len = tokens ? (d->seqlen > 0 ? d->seqlen : 1) : 1;
  // element counts with headroom for padded tiles, byte sizes and strides
  int64_t hp, row, t, bh;
  if (!mul_ok(d->heads, d->headdim, &hp) || !mul_ok(d->groups, d->dstate, &row)) return S6_ERR_SHAPE;
  if (hp > INT32_MAX / 256 || row > INT32_MAX / 256) return S6_ERR_SHAPE;  // one token's row in 32 bits
  if (!mul_ok(d->batch, hp, &bh) || !mul_ok(bh, len, &t) || !mul_ok(t, 1024, &t)) return S6_ERR_SHAPE;
  if (!mul_ok(bh, 128 * 1024, &t) || !mul_ok(d->batch, row, &t) || !mul_ok(t, len, &t) || !mul_ok(t, 4096, &t))
    return S6_ERR_SHAPE;
  if (bh / d->headdim > INT32_MAX / 4 || len > INT32_MAX / 4) return S6_ERR_SHAPE;  // grid and token indices
  const int64_t str[] = {d->x_batch, d->x_token, d->delta_batch, d->delta_token,
                         d->b_batch, d->b_token, d->c_batch, d->c_token};
  for (int i = 0; i < 8; ++i) {
    const bool token = i & 1;
    if (token && !tokens) continue;
    if (!has_delta && (i == 2 || i == 3)) continue;
    if (str[i] < 0) return S6_ERR_SHAPE;
    if (!mul_ok(str[i], token ? len : d->batch, &t) || !mul_ok(t, 8, &t)) return S6_ERR_SHAPE;
  }
  return S6_OK;
}

}  // namespace s6i

using namespace s6i;

extern "C" int s6_heads_state_update(const s6_heads_dims* d, int in_dtype, int flags, float* h, const void* x,
                                     const void* delta, const float* delta_bias, const float* A, const void* Bm,
                                     const void* Cm, const float* D, void* y, void* stream) {
  const int rc = check_heads(d, in_dtype, flags, delta != nullptr, delta_bias != nullptr, false);
  if (rc) return rc;
  if (d->batch == 0 || d->heads == 0) return S6_OK;
  if (!h || !x || !A || !Bm || !Cm || !y) return S6_ERR_NULL;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4;
  const void* ins[] = {x, delta, Bm, Cm, y};
  for (const void* p : ins)
    if (!aligned(p, esz)) return S6_ERR_ALIGN;
  const void* f32s[] = {h, delta_bias, A, D};
  for (const void* p : f32s)
    if (!aligned(p, 4)) return S6_ERR_ALIGN;
  const bool vec = d->dstate % 4 == 0 && aligned(h, 16) && aligned(Bm, 4 * esz) && aligned(Cm, 4 * esz) &&
                   d->b_batch % 4 == 0 && d->c_batch % 4 == 0;
  StepHeadsArgs a;
  a.h = h; a.x = x; a.delta = delta; a.dbias = delta_bias; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.y = y;
  a.softplus = (flags & S6_DELTA_SOFTPLUS) != 0;
  a.unit = (flags & S6_UNIT_INPUT) != 0;
  a.heads = (int)d->heads; a.headdim = (int)d->headdim; a.hpg = (int)(d->heads / d->groups); a.dstate = (int)d->dstate;
  a.x_batch = d->x_batch; a.delta_batch = d->delta_batch; a.b_batch = d->b_batch; a.c_batch = d->c_batch;
  const int64_t pairs = d->batch * d->heads;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return in_dtype == S6_BF16 ? dispatch_step<uint16_t>(a, pairs, vec, st) : dispatch_step<float>(a, pairs, vec, st);
}
