// heads_state.hip -- the state walk of the multi-head scan: the state's
// recurrence alone, forward in time, or that of its adjoint, backward in
// time, chunk by chunk of 64 tokens:
//
//   forward   S <- e^{c_Q} S + sum_s (w_s e^{c_Q - c_s} x_s) B_s^T
//   backward  L <- e^{c_Q} L + sum_t (e^{c_t} dy_t) C_t^T
//
// (c: running sum of the log decays in the chunk, c_Q its last).  Used for
// segments of few long rows (their end states from zero, then the fold), and
// by the backward, which stores the state entering every block of tokens.
//
// A workgroup of four waves owns one row (64 channels of a head): wave w the
// channel tiles 2 (w & 1), + 1 and half of the state columns, in registers.
// The scaled inputs enter as three bf16 parts, so the state is good to fp32
// accumulation.
//
// For the backward it is bound by HBM: 8 x 2048 tokens of 80 heads of 64, N
// 128: 0.34 GB read (x, dy) and 0.67 GB of states stored in both directions in
// 231 us, 4.4 TB/s.  Over segments (nothing stored) by a chunk's latency, as the
// scan: 65536 tokens of 24 heads of 64, N 64: 84 - 100 us.  The channel tiles of a
// wave pair lie side by side in the stored planes, 16 bytes per lane and store.
#include "heads_kernel.h"

namespace s6i {

namespace {

// Tokens per stored block: 128 (bf16) or 64 (fp32), see heads_bwd.hip.
template <typename In>
constexpr int kBlockTokens = sizeof(In) == 2 ? 128 : 64;

template <typename In, int NT, bool VEC>
__global__ __launch_bounds__(256, sizeof(In) == 2 ? (VEC ? 3 : 2) : 1) void s6_heads_state_kernel(HeadsArgs a, int mode) {
  constexpr int NW = NT / 32;  // state tiles of 16 columns per wave and channel tile
  using XT = ColTile<In, kTP>;
  using BT = ColTile<In, NT>;
  __shared__ __align__(16) In xmem[XT::size(kHQ)];
  __shared__ __align__(16) In bmem[BT::size(kHQ)];
  const XT xs{xmem};
  const BT bs{bmem};
  __shared__ __align__(16) float wt[kHQ];
  __shared__ float total_s;
  const HeadRow hr = head_row(a, a.row0 + blockIdx.x);
  const int64_t nrows = a.rows;
  const int dir = blockIdx.z;
  const int64_t seg = mode == 0 && dir ? blockIdx.y + 1 : blockIdx.y;
  const int lane = threadIdx.x & 63, wv = wave_index(), g = lane >> 4, c = lane & 15;
  const int pp = wv & 1, nh = wv >> 1;
  const int p0 = hr.pt * kTP, pleft = a.headdim - p0;
  const int64_t t_lo = seg * a.seg_len;
  const int64_t t_hi = t_lo + a.seg_len < a.L ? t_lo + a.seg_len : a.L;
  const int64_t nch = (t_hi - t_lo + kHQ - 1) / kHQ;
  const int64_t hp = (int64_t)a.heads * a.headdim;
  const In* X;
  const In* B;
  int64_t xt, bt;
  if (dir == 0) {
    X = static_cast<const In*>(a.x) + hr.b * a.x_batch + (int64_t)hr.hd * a.headdim + p0;
    B = static_cast<const In*>(a.Bm) + hr.b * a.b_batch + (int64_t)hr.grp * a.dstate;
    xt = a.x_token; bt = a.b_token;
  } else {
    X = static_cast<const In*>(a.dy) + hr.b * a.L * hp + (int64_t)hr.hd * a.headdim + p0;
    B = static_cast<const In*>(a.Cm) + hr.b * a.c_batch + (int64_t)hr.grp * a.dstate;
    xt = hp; bt = a.c_token;
  }
  const In* dl = a.delta ? static_cast<const In*>(a.delta) + hr.b * a.d_batch + hr.hd : nullptr;
  const float bias = a.dbias ? a.dbias[hr.hd] : 0.0f;
  const float a2 = a.A[hr.hd] * kLog2e;

  // state tiles: rows p = 16 (2 pp + j) + 4 g + r, column n = 16 (nh NW + i) + c
  f32x4 T[NW][2];
  const float* init = nullptr;
  if (mode == 1 && a.hin)
    init = a.hin + ((dir * a.nseg + seg) * nrows + hr.row) * (int64_t)(kTP * NT);
  const float* user = mode == 1 && !a.hin ? (dir ? a.dh_last : a.h0) : nullptr;
  const int64_t srow = ((hr.b * a.heads + hr.hd) * (int64_t)a.headdim + p0);
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int p = 16 * (2 * pp + j) + 4 * g + r, n = 16 * (nh * NW + i) + c;
        float v = 0.0f;
        if (init)
          v = init[p * NT + n];
        else if (user && p < pleft && n < a.dstate)
          v = user[(srow + p) * a.dstate + n];
        T[i][j][r] = v;
      }

  int x_col = XT::col_lane(g, c), b_col = BT::col_lane(g, c);  // lane parts of the LDS addresses

  TileRegs<In, kHQ, kTP, 256, VEC> xr;
  TileRegs<In, kHQ, NT, 256, VEC> br;
  In draw = In(0);  // as loaded: a conversion here would wait for every load before it
  auto issue = [&](int64_t k) {
    const int64_t t0 = t_lo + k * kHQ;
    const int rows = k < 0 || k >= nch ? 0 : (int)(t_hi - t0 < kHQ ? t_hi - t0 : kHQ);
    xr.load(X + t0 * xt, xt, rows, pleft < kTP ? pleft : kTP);
    br.load(B + t0 * bt, bt, rows, a.dstate);
    if (wv == 0 && dl) load_step<In, VEC>(draw, dl + t0 * a.d_token, a.d_token, lane, rows);
  };
  const int64_t first = dir ? nch - 1 : 0, step = dir ? -1 : 1;
  issue(first);
  float sum = 0.0f;
  constexpr int kPerBlock = kBlockTokens<In> / kHQ;
  for (int64_t i = 0, k = first; i < nch; ++i, k += step) {
    const int64_t t0 = t_lo + k * kHQ;
    const int rows = (int)(t_hi - t0 < kHQ ? t_hi - t0 : kHQ);
    // the state entering a stored block, from its near end
    const bool enter = dir ? ((k + 1) % kPerBlock == 0 || k == nch - 1) : k % kPerBlock == 0;
    if (mode == 1 && a.planes && enter) {
      const int64_t blk = t0 / kBlockTokens<In>, nblk = (a.L + kBlockTokens<In> - 1) / kBlockTokens<In>;
      // operand order: [state tile][channel half][four of eight][lane][4], see heads_bwd.hip
      float* pl = a.planes + ((dir * nblk + blk) * nrows + hr.row) * (int64_t)(kTP * NT);
#pragma unroll
      for (int q = 0; q < NW; ++q) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float f[4] = {T[q][j][0], T[q][j][1], T[q][j][2], T[q][j][3]};
          store_vec<float, 4>(pl + ((((nh * NW + q) * 2 + pp) * 2 + j) * 64 + lane) * 4, f);
        }
      }
    }
    xr.mask(rows, pleft < kTP ? pleft : kTP);
    br.mask(rows, a.dstate);
    xr.store(xs);
    br.store(bs);
    if (wv == 0) {
      const bool on = lane < rows;
      const float s = on ? step_of(a, to_f32(draw), bias) : 0.0f;
      const LogSum cs = log_scan(on ? clamp_log2(s * a2) : 0.0f), cq = last_lane(cs);
      const float w = on ? (a.unit ? 1.0f : s) : 0.0f;
      wt[lane] = dir ? fast_exp2(cs.hi + cs.lo) : w * decay_between(cq, cs);
      if (lane == 0) total_s = cq.hi + cq.lo;
    }
    __syncthreads();
    issue(k + step);
    const float cq = total_s;
    sum += cq;
    const float dec = fast_exp2(cq);
#pragma unroll
    for (int q = 0; q < NW; ++q)
#pragma unroll
      for (int j = 0; j < 2; ++j) T[q][j] *= dec;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const float4 w0 = *reinterpret_cast<const float4*>(wt + 32 * kk + 4 * g);
      const float4 w1 = *reinterpret_cast<const float4*>(wt + 32 * kk + 16 + 4 * g);
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      Whole<In> xd[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const Frag<In> xf = xs.col(x_col, 2 * pp + j, kk, g, c);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = frag_f32(xf, e) * w[e];
        to_whole(f, xd[j]);
      }
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        const Frag<In> bf = bs.col(b_col, nh * NW + q, kk, g, c);
#pragma unroll
        for (int i = Whole<In>::kParts - 1; i >= 0; --i)
#pragma unroll
          for (int j = 0; j < 2; ++j) T[q][j] = mma(xd[j].part[i], bf, T[q][j]);
      }
    }
    __syncthreads();
  }

  if (mode == 0) {
    const int64_t at = (dir * a.nseg + seg) * nrows + hr.row;
    float* o = a.agg + at * (int64_t)(kTP * NT);
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) o[(16 * (2 * pp + j) + 4 * g + r) * NT + 16 * (nh * NW + i) + c] = T[i][j][r];
    if (threadIdx.x == 0) a.sd[at] = sum;
  } else if (dir == 1 && a.dh0 && seg == 0) {
#pragma unroll
    for (int i = 0; i < NW; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int p = 16 * (2 * pp + j) + 4 * g + r, n = 16 * (nh * NW + i) + c;
          if (p < pleft && n < a.dstate) a.dh0[(srow + p) * a.dstate + n] = T[i][j][r];
        }
  }
}

// hin[first] = h0 (dh_last), hin[next] = 2^sd hin + agg, four values per
// thread; the aggregates do not depend on the chain, so eight of them are
// loaded before each batch of it.
template <int NT>
__global__ __launch_bounds__(256) void s6_heads_fold_kernel(HeadsArgs a, int64_t nrows) {  // (few rows: one launch)
  const int64_t row = blockIdx.x;
  const int dir = blockIdx.z;
  const int e = (blockIdx.y * 256 + threadIdx.x) * 4;  // in the row's 64 x NT tile
  const int p = e / NT, n = e % NT;
  const HeadRow hr = head_row(a, row);
  const float* user = dir ? a.dh_last : a.h0;
  float v[4] = {0, 0, 0, 0};
  if (user && hr.pt * kTP + p < a.headdim) {
    const float* u = user + ((hr.b * a.heads + hr.hd) * (int64_t)a.headdim + hr.pt * kTP + p) * a.dstate + n;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (n + j < a.dstate) v[j] = u[j];
  }
  const int64_t tile = (int64_t)kTP * NT;
  // segment i of the walk is segment i in time, or counted from the end
  auto at = [&](int64_t i) { return (dir * a.nseg + (dir ? a.nseg - 1 - i : i)) * nrows + row; };
  for (int64_t s = 0; s < a.nseg; s += 8) {
    float b[8][4], d[8];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (s + k < a.nseg - 1) {
        load_vec<float, 4>(a.agg + at(s + k) * tile + e, b[k]);
        d[k] = a.sd[at(s + k)];
      }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (s + k < a.nseg) store_vec<float, 4>(a.hin + at(s + k) * tile + e, v);
      if (s + k < a.nseg - 1) {
        const float f = fast_exp2(d[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_fmaf(f, v[j], b[k][j]);
      }
    }
  }
}

template <typename In, int NT>
int launch_state_t(HeadsArgs a, const HeadsPlan& p, int mode, int dirs, hipStream_t st) {
  for (a.row0 = 0; a.row0 < p.rows; a.row0 += kMaxBlocks) {
    const int64_t n = p.rows - a.row0 < kMaxBlocks ? p.rows - a.row0 : kMaxBlocks;
    const dim3 grid((unsigned)n, (unsigned)(mode == 0 ? a.nseg - 1 : a.nseg), (unsigned)dirs);
    if (p.vec)
      hipLaunchKernelGGL((s6_heads_state_kernel<In, NT, true>), grid, dim3(256), 0, st, a, mode);
    else
      hipLaunchKernelGGL((s6_heads_state_kernel<In, NT, false>), grid, dim3(256), 0, st, a, mode);
    S6_HIP(hipGetLastError(), "s6_heads_state_kernel launch");
  }
  return S6_OK;
}

template <typename In>
int launch_state_in(const HeadsArgs& a, const HeadsPlan& p, int mode, int dirs, hipStream_t st) {
  if (p.NT == 32) return launch_state_t<In, 32>(a, p, mode, dirs, st);
  if (p.NT == 64) return launch_state_t<In, 64>(a, p, mode, dirs, st);
  return launch_state_t<In, 128>(a, p, mode, dirs, st);
}

}  // namespace

int launch_heads_state(int in_dtype, const HeadsArgs& a, const HeadsPlan& p, int mode, int dirs, hipStream_t st) {
  return in_dtype == S6_BF16 ? launch_state_in<uint16_t>(a, p, mode, dirs, st)
                             : launch_state_in<float>(a, p, mode, dirs, st);
}

int launch_heads_fold(const HeadsArgs& a, const HeadsPlan& p, int dirs, hipStream_t st) {
  const dim3 grid((unsigned)p.rows, (unsigned)(kTP * p.NT / 1024), (unsigned)dirs);
  if (p.NT == 32) hipLaunchKernelGGL((s6_heads_fold_kernel<32>), grid, dim3(256), 0, st, a, p.rows);
  else if (p.NT == 64) hipLaunchKernelGGL((s6_heads_fold_kernel<64>), grid, dim3(256), 0, st, a, p.rows);
  else hipLaunchKernelGGL((s6_heads_fold_kernel<128>), grid, dim3(256), 0, st, a, p.rows);
  S6_HIP(hipGetLastError(), "s6_heads_fold_kernel launch");
  return S6_OK;
}

}  // namespace s6i
