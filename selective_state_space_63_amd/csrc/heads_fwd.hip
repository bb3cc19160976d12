// heads_fwd.hip -- the multi-head scan over whole sequences
// (s6_heads_scan_fwd) and the launch plan shared by the heads entry points.
//
// In chunks of Q = 64 tokens, c the running sum of the log decays s A in the
// chunk:
//   y_t = sum_{s<=t} (C_t . B_s) e^{c_t - c_s} w_s x_s + e^{c_t} S C_t + D x_t
//   S  <- e^{c_Q} S + sum_s (w_s e^{c_Q - c_s} x_s) B_s^T
// so each chunk is four matrix products: the Gram matrix C B^T (its lower
// half), its decayed form times x, the entering state times C, and the chunk's
// own part of the state.  x is read and y written once; the state never
// leaves the registers.
//
// A workgroup of four waves owns one row (64 channels of one head of one
// sequence) and walks it; wave w owns channels 16 w .. 16 w + 15 of the
// output and of the state (NT x 16 in registers, rows n).  Results are made
// transposed (channels x tokens), so that a lane stores four channels of one
// token, the decay of its token is one scalar per lane, and the state's
// registers are the operand of the product with C as they are.  The decayed
// Gram tiles are shared out among the waves and meet in LDS in operand order.
//
// Roundings (bf16 inputs): the decayed Gram matrix and the state's copy for
// the product with C enter as two bf16 parts (within 2^-17), so that y meets one
// rounding, its own; the diagonal (a token's own input) stays in fp32 with the
// skip; the inputs of the state itself enter in full, as three bf16 parts.
//
// What bounds it: the latency of a chunk's chain (stage -> Gram -> y -> state,
// three barriers), not a unit: at 8 x 2048 tokens of 80 heads of 64, N 128,
// 235 us in a queue of its own (245 - 270 us between other kernels), 1.6 TB/s
// of the 6.2 TB/s that a copy reaches, with the vector units 44 % and the
// matrix units 24 % busy and LDS 31 %; a chunk takes 7.3 us with three
// workgroups on a CU.  So what counts is workgroups per CU: 168 VGPRs and 52.5
// KB of LDS let three in.  The second parts in y cost 11 % of the scan with one
// (10 % at N 64, 2 % for few long rows).  Measured and not kept: Gram tiles of a
// wave side by side (+6 %), Gram tiles formed once per group by a launch of their
// own (+2 %, registers), the state's part of y beside the Gram tiles instead of
// behind them (+1 to +4 %), four workgroups per CU (spills; at N 64 +6 %).
#include "heads_kernel.h"

namespace s6i {

namespace {

// The decayed Gram matrix in LDS: the ten tiles J <= I of 256 values, in operand
// order: two tiles J = 2 kk, 2 kk + 1 per operand, or the diagonal tile of an even
// I alone (what is right of it is 0).
constexpr int kGram = 2560;
__device__ __forceinline__ int gram_at(int I, int kk) { return (I == 0 ? 0 : I == 1 ? 256 : I == 2 ? 768 : 1536) + 512 * kk; }
template <typename In>
__device__ __forceinline__ Frag<In> gram_frag(const In* p, int I, int kk, int lane) {
  if (kk < I / 2 || (I & 1)) return lane_frag(p + gram_at(I, kk), lane);
  float f[4], e[8];
  load_vec<In, 4>(p + gram_at(I, kk) + 4 * lane, f);
#pragma unroll
  for (int r = 0; r < 8; ++r) e[r] = r < 4 ? f[r] : 0.0f;
  Frag<In> o;
  to_frag(e, o);
  return o;
}

// Offsets in LDS (bytes).
template <typename In, int NT>
struct ScanLds {
  using XT = ColTile<In, kTP>;
  using BT = ColTile<In, NT>;
  using CT = RowTile<In, NT>;
  static constexpr int xs = 0;
  static constexpr int bs = xs + XT::size(kHQ) * (int)sizeof(In);
  static constexpr int cm = bs + BT::size(kHQ) * (int)sizeof(In);
  static constexpr int pf = cm + CT::size(kHQ) * (int)sizeof(In);
  static constexpr int tok = pf + (sizeof(In) == 2 ? 2 : 1) * kGram * (int)sizeof(In);
  static constexpr int dg = tok + 2 * 4 * kHQ * 4;
  static constexpr int bad = dg + kHQ * 4;
  static constexpr int total = bad + kTP * 4;
};
// Three workgroups of bf16 fit a CU (LDS is given out in pieces of 1280 bytes).
static_assert(3 * ((ScanLds<uint16_t, 128>::total + 1279) / 1280 * 1280) <= 163840, "LDS");

template <typename In, int NT, bool VEC>
__global__ __launch_bounds__(256, sizeof(In) == 2 ? (VEC ? 3 : 2) : 1) void s6_heads_scan_kernel(HeadsArgs a) {
  constexpr int NQ = NT / 16, NK = NT / 32;
  using L = ScanLds<In, NT>;
  extern __shared__ __align__(16) char lds[];
  const typename L::XT xs{reinterpret_cast<In*>(lds + L::xs)};
  const typename L::BT bs{reinterpret_cast<In*>(lds + L::bs)};
  const typename L::CT cm{reinterpret_cast<In*>(lds + L::cm)};
  In* pf = reinterpret_cast<In*>(lds + L::pf);             // decayed Gram matrix; bf16: two parts of kGram
  float* tok = reinterpret_cast<float*>(lds + L::tok);     // per-token values, two chunks' worth
  float* dg = reinterpret_cast<float*>(lds + L::dg);       // the Gram matrix's diagonal times the weights
  int* bad = reinterpret_cast<int*>(lds + L::bad);         // first token whose input is not finite
  // consecutive workgroups go to the 8 XCDs in turn: give each XCD a run of
  // rows, whose B and C come through one L2
  const uint32_t here = gridDim.x;
  const uint32_t rid = here % 8 == 0 ? (blockIdx.x % 8) * (here / 8) + blockIdx.x / 8 : blockIdx.x;
  const HeadRow hr = head_row(a, a.row0 + rid);
  const int64_t seg = blockIdx.y;
  const int lane = threadIdx.x & 63, wv = wave_index(), g = lane >> 4, c = lane & 15;
  const int p0 = hr.pt * kTP, pleft = a.headdim - p0;
  const int64_t t_lo = seg * a.seg_len;
  const int64_t t_hi = t_lo + a.seg_len < a.L ? t_lo + a.seg_len : a.L;
  const int64_t hp = (int64_t)a.heads * a.headdim;
  const In* X = static_cast<const In*>(a.x) + hr.b * a.x_batch + (int64_t)hr.hd * a.headdim + p0;
  const In* B = static_cast<const In*>(a.Bm) + hr.b * a.b_batch + (int64_t)hr.grp * a.dstate;
  const In* C = static_cast<const In*>(a.Cm) + hr.b * a.c_batch + (int64_t)hr.grp * a.dstate;
  const In* dl = a.delta ? static_cast<const In*>(a.delta) + hr.b * a.d_batch + hr.hd : nullptr;
  In* Y = static_cast<In*>(a.y) + hr.b * a.L * hp + (int64_t)hr.hd * a.headdim + p0;
  const float bias = a.dbias ? a.dbias[hr.hd] : 0.0f;
  const float a2 = a.A[hr.hd] * kLog2e;
  const float dsk = a.D ? a.D[hr.hd] : 0.0f;

  if (threadIdx.x < kTP) bad[threadIdx.x] = kHQ;

  // state tiles: rows n = 16 q + 4 g + r, column p = 16 wv + c
  f32x4 S[NQ];
  const int64_t srow = (hr.b * a.heads + hr.hd) * (int64_t)a.headdim + p0;
  const int ps = 16 * wv + c;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    S[q] = f32x4{0, 0, 0, 0};
    const int n = 16 * q + 4 * g;
    if (a.hin) {
      float v[4];
      load_vec<float, 4>(a.hin + (seg * a.rows + hr.row) * (int64_t)(kTP * NT) + ps * NT + n, v);
#pragma unroll
      for (int r = 0; r < 4; ++r) S[q][r] = v[r];
    } else if (a.h0 && ps < pleft) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < a.dstate) S[q][r] = a.h0[(srow + ps) * a.dstate + n + r];
    }
  }

  TileRegs<In, kHQ, kTP, 256, VEC> xr;
  TileRegs<In, kHQ, NT, 256, VEC> br, cr;
  auto rows_at = [&](int64_t t0) { return t0 >= t_hi ? 0 : (int)(t_hi - t0 < kHQ ? t_hi - t0 : kHQ); };
  auto issue = [&](int64_t t0) {
    const int rows = rows_at(t0);
    xr.load(X + t0 * a.x_token, a.x_token, rows, pleft < kTP ? pleft : kTP);
    br.load(B + t0 * a.b_token, a.b_token, rows, a.dstate);
    cr.load(C + t0 * a.c_token, a.c_token, rows, a.dstate);
  };
  // The last wave (it has the fewest Gram tiles) forms the tokens' decays and
  // weights a chunk ahead, from steps loaded two chunks ahead: running log2
  // decay in two parts, input weight, weight decayed to the chunk's end.
  In draw = In(0);  // as loaded: a conversion here would wait for every load before it
  auto issue_step = [&](int64_t t0) {
    if (wv == 3 && dl) load_step<In, VEC>(draw, dl + t0 * a.d_token, a.d_token, lane, rows_at(t0));
  };
  auto decays = [&](int64_t t0, int buf) {
    if (wv != 3) return;
    const bool on = lane < rows_at(t0);
    const float s = on ? step_of(a, to_f32(draw), bias) : 0.0f;
    const LogSum v = log_scan(on ? clamp_log2(s * a2) : 0.0f);
    const float w = on ? (a.unit ? 1.0f : s) : 0.0f;
    float* o = tok + buf * 4 * kHQ;
    o[lane] = v.hi;
    o[kHQ + lane] = v.lo;
    o[2 * kHQ + lane] = w;
    o[3 * kHQ + lane] = w * decay_between(last_lane(v), v);
  };
  issue_step(t_lo);
  issue(t_lo);
  decays(t_lo, 0);
  issue_step(t_lo + kHQ);
  __syncthreads();
  int buf = 0;
  // a lane's place in a tile of y: channels 16 wv + 4 g .., token c
  const uint32_t y_row = (uint32_t)hp * (uint32_t)sizeof(In);
  const uint32_t y_off =
      16 * wv + 4 * g < pleft ? (uint32_t)c * y_row + (uint32_t)(16 * wv + 4 * g) * (uint32_t)sizeof(In) : kNowhere;
  // lane parts of the LDS addresses; x's column tile is the wave's own
  int b_row = L::BT::row_lane(g, c), b_col = L::BT::col_lane(g, c), c_row = L::CT::row_lane(g, c);
  const int x_col = L::XT::col_lane(g, c);
  Four<In> yv[4];  // a chunk's y: channels 16 wv + 4 g .., token 16 I + c

  auto put_y = [&](int64_t t0) {
    const int rows = rows_at(t0);
    In* const base = Y + t0 * hp;
    if constexpr (VEC) {  // rows past the sequence and channels past the head are dropped
      const __amdgpu_buffer_rsrc_t yb =
          buffer_of(base, (uint32_t)(rows - 1) * y_row + (uint32_t)(pleft < kTP ? pleft : kTP) * (uint32_t)sizeof(In));
#pragma unroll
      for (int I = 0; I < 4; ++I) yv[I].store(yb, y_off == kNowhere ? kNowhere : y_off + (uint32_t)(16 * I) * y_row);
    } else {
      const int p = 16 * wv + 4 * g;
#pragma unroll
      for (int I = 0; I < 4; ++I)
        if (16 * I + c < rows) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (p + r < pleft) base[(16 * I + c) * hp + p + r] = yv[I].get(r);
        }
    }
  };
  for (int64_t t0 = t_lo; t0 < t_hi; t0 += kHQ, buf ^= 1) {
    const int rows = rows_at(t0);
    // the units' XORs are done in every turn: their results kept over it would
    // cost a workgroup per CU
    asm volatile("" : "+v"(b_row), "+v"(b_col), "+v"(c_row));
    const float* cs = tok + buf * 4 * kHQ;
    const float *cl = cs + kHQ, *ww = cs + 2 * kHQ, *wd = cs + 3 * kHQ;
    // An input that is not finite would reach earlier tokens through the
    // zeros of the Gram matrix (0 x inf): it is taken out here and its channel
    // set to NaN from its token on.
    const int cols = pleft < kTP ? pleft : kTP;
    xr.mask(rows, cols);
    br.mask(rows, a.dstate);
    cr.mask(rows, a.dstate);
    xr.clean(bad);
    xr.store(xs);
    br.store(bs);
    cr.store(cm);
    __syncthreads();
    issue(t0 + kHQ);
    decays(t0 + kHQ, buf ^ 1);
    issue_step(t0 + 2 * kHQ);

    // decayed Gram tiles (rows s of tile J, columns t of tile I), J <= I
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const int id = 4 * k + wv;
      if (k < 2 || id < 10) {
        int I = id >= 6 ? 3 : id >= 3 ? 2 : id >= 1 ? 1 : 0;
        I = __builtin_amdgcn_readfirstlane(I);
        asm volatile("" : "+s"(I));  // addresses of the tile are formed here, not kept over the loop
        const int J = id - I * (I + 1) / 2;
        f32x4 G = {0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < NK; ++kk)
          G = mma(bs.row(b_row, 16 * J, kk), cm.row(c_row, 16 * I, kk), G);
        const float ct = cs[16 * I + c], lt = cl[16 * I + c];
        const float4 cv = *reinterpret_cast<const float4*>(cs + 16 * J + 4 * g);
        const float4 lv = *reinterpret_cast<const float4*>(cl + 16 * J + 4 * g);
        const float4 wv4 = *reinterpret_cast<const float4*>(ww + 16 * J + 4 * g);
        const float cj[4] = {cv.x, cv.y, cv.z, cv.w}, lj[4] = {lv.x, lv.y, lv.z, lv.w};
        const float wj[4] = {wv4.x, wv4.y, wv4.z, wv4.w};
        float p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
          p[r] = I != J || c > 4 * g + r ? G[r] * (decay_between(ct, lt, cj[r], lj[r]) * wj[r]) : 0.0f;
        if (I == J) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (c == 4 * g + r) dg[16 * I + c] = G[r] * wj[r];
        }
        In* at = pf + gram_at(I, J >> 1) + (I == J && !(I & 1) ? 4 * lane : 8 * lane + 4 * (J & 1));
        if constexpr (sizeof(In) == 2) {
          Four<In> hi;
          hi.split(p);
          hi.put(at);
          store_vec<In, 4>(at + kGram, p);
        } else {
          store_vec<In, 4>(at, p);
        }
      }
    }
    __syncthreads();

    Frag<In> xf[2];
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) xf[kk] = xs.col(x_col, wv, kk, g, c);
    {
      f32x4 out[4];
#pragma unroll
      for (int I = 0; I < 4; ++I) out[I] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int kk = 0; kk < NK; ++kk) {
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = S[2 * kk + (e >> 2)][e & 3];
        Pair<In> sf;
        to_pair(f, sf);
#pragma unroll
        for (int I = 0; I < 4; ++I) out[I] = mma_pair(sf, cm.row(c_row, 16 * I, kk), out[I]);
      }
      __builtin_amdgcn_sched_barrier(0);  // (mixed with what follows it would spill)
      const bool dirty = __builtin_amdgcn_ballot_w64(bad[lane] != kHQ) != 0;
      const int p = 16 * wv + 4 * g;
#pragma unroll
      for (int I = 0; I < 4; ++I) {
        f32x4 acc = out[I] * fast_exp2(cs[16 * I + c] + cl[16 * I + c]);
#pragma unroll
        for (int kk = 0; kk <= I / 2; ++kk) {
          Pair<In> gm;
          gm.hi = gram_frag(pf, I, kk, lane);
          if constexpr (sizeof(In) == 2) gm.lo = gram_frag(pf + kGram, I, kk, lane);
          acc = mma_pair(xf[kk], gm, acc);
        }
        float xv[4], o[4];
        xs.four(16 * I + c, 4 * wv + g, xv);
        // a token's own input enters in fp32, with the skip: it is the largest
        // term of heads that forget fast, which would meet two roundings
        const float own = dsk + dg[16 * I + c];
#pragma unroll
        for (int r = 0; r < 4; ++r) o[r] = __builtin_fmaf(own, xv[r], acc[r]);
        yv[I].set(o);
      }
      if (dirty) {
#pragma unroll
        for (int I = 0; I < 4; ++I) {
          float o[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) o[r] = 16 * I + c >= bad[p + r] ? __builtin_nanf("") : to_f32(yv[I].get(r));
          yv[I].set(o);
        }
      }
      if (dirty && bad[ps] < kHQ) {
#pragma unroll
        for (int q = 0; q < NQ; ++q) S[q] = f32x4{1, 1, 1, 1} * __builtin_nanf("");
      }
    }

    put_y(t0);
    const float dec = fast_exp2(cs[kHQ - 1] + cl[kHQ - 1]);
#pragma unroll
    for (int q = 0; q < NQ; ++q) S[q] *= dec;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const float4 w0 = *reinterpret_cast<const float4*>(wd + 32 * kk + 4 * g);
      const float4 w1 = *reinterpret_cast<const float4*>(wd + 32 * kk + 16 + 4 * g);
      const float w[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = frag_f32(xf[kk], e) * w[e];
      Whole<In> xd;
      to_whole(f, xd);
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const Frag<In> bf = bs.col(b_col, q, kk, g, c);
#pragma unroll
        for (int i = Whole<In>::kParts - 1; i >= 0; --i) S[q] = mma(bf, xd.part[i], S[q]);
      }
    }
    __syncthreads();
  }

  if (a.h_last && seg == a.nseg - 1 && ps < pleft) {
    float* o = a.h_last + (srow + ps) * a.dstate;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int n = 16 * q + 4 * g;
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < a.dstate) o[n + r] = S[q][r];
    }
  }
}

template <typename In, int NT, bool VEC>
int launch_scan_v(HeadsArgs a, const HeadsPlan& p, hipStream_t st) {
  const auto kern = s6_heads_scan_kernel<In, NT, VEC>;
  constexpr int lds = ScanLds<In, NT>::total;
  if constexpr (lds > 65536)
    S6_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds),
           "s6_heads_scan_kernel LDS size");
  for (a.row0 = 0; a.row0 < p.rows; a.row0 += kMaxBlocks) {
    const int64_t n = p.rows - a.row0 < kMaxBlocks ? p.rows - a.row0 : kMaxBlocks;
    hipLaunchKernelGGL(kern, dim3((unsigned)n, (unsigned)a.nseg), dim3(256), lds, st, a);
    S6_HIP(hipGetLastError(), "s6_heads_scan_kernel launch");
  }
  return S6_OK;
}
template <typename In, int NT>
int launch_scan_n(const HeadsArgs& a, const HeadsPlan& p, hipStream_t st) {
  return p.vec ? launch_scan_v<In, NT, true>(a, p, st) : launch_scan_v<In, NT, false>(a, p, st);
}
template <typename In>
int launch_scan_in(const HeadsArgs& a, const HeadsPlan& p, hipStream_t st) {
  if (p.NT == 32) return launch_scan_n<In, 32>(a, p, st);
  if (p.NT == 64) return launch_scan_n<In, 64>(a, p, st);
  return launch_scan_n<In, 128>(a, p, st);
}

// Segment states of the forward in the workspace.
struct FwdWs {
  int64_t nseg, seg_len;
  size_t agg, sd, hin, total;
};
FwdWs fwd_ws(const s6_heads_dims& d, const HeadsPlan& p) {
  FwdWs o;
  heads_segments(p.rows, d.seqlen, kHQ, &o.nseg, &o.seg_len);
  o.agg = o.sd = o.hin = o.total = 0;
  if (o.nseg > 1) {
    const size_t tile = (size_t)p.rows * kTP * p.NT * sizeof(float);
    o.sd = up256((size_t)o.nseg * tile);
    o.hin = o.sd + up256((size_t)o.nseg * p.rows * sizeof(float));
    o.total = o.hin + up256((size_t)o.nseg * tile);
  }
  return o;
}

}  // namespace

HeadsPlan heads_plan(const s6_heads_dims& d, int in_dtype, const void* x, const void* Bm, const void* Cm,
                     const void* dy) {
  HeadsPlan p;
  p.NT = d.dstate > 64 ? 128 : d.dstate > 32 ? 64 : 32;
  p.ptiles = (d.headdim + kTP - 1) / kTP;
  p.rows = d.batch * d.heads * p.ptiles;
  const int64_t u = in_dtype == S6_BF16 ? 8 : 4;  // elements of 16 bytes
  p.vec = d.headdim % 8 == 0 && d.dstate % 8 == 0 && d.x_batch % u == 0 && d.x_token % u == 0 && d.b_batch % u == 0 &&
          d.b_token % u == 0 && d.c_batch % u == 0 && d.c_token % u == 0 && aligned(x, 16) && aligned(Bm, 16) &&
          aligned(Cm, 16) && aligned(dy, 16);
  // offsets within a tile of up to 128 rows in 32 bits
  const int64_t hp = d.heads * d.headdim, gn = d.groups * d.dstate;
  const int64_t strides[] = {d.x_token, d.b_token, d.c_token, d.delta_token, hp};
  for (int64_t s : strides) p.vec = p.vec && s < (int64_t(1) << 31) / (128 * 4);
  // a tile's buffer ends with its last token: rows past it must lie past that
  // end (not so where tokens share their row, as in a broadcast)
  p.vec = p.vec && d.x_token >= hp && d.b_token >= gn && d.c_token >= gn;
  return p;
}

HeadsArgs heads_args(const s6_heads_dims& d, const HeadsPlan& p, int flags, const void* x, const void* delta,
                     const float* dbias, const float* A, const void* Bm, const void* Cm, const float* D,
                     const float* h0) {
  HeadsArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.delta = delta; a.dbias = dbias; a.A = A; a.Bm = Bm; a.Cm = Cm; a.D = D; a.h0 = h0;
  a.softplus = (flags & S6_DELTA_SOFTPLUS) != 0;
  a.unit = (flags & S6_UNIT_INPUT) != 0;
  a.heads = (int)d.heads; a.headdim = (int)d.headdim; a.ptiles = (int)p.ptiles; a.hpg = (int)(d.heads / d.groups);
  a.dstate = (int)d.dstate;
  a.batch = d.batch; a.L = d.seqlen; a.rows = p.rows;
  a.x_batch = d.x_batch; a.x_token = d.x_token; a.d_batch = d.delta_batch; a.d_token = d.delta_token;
  a.b_batch = d.b_batch; a.b_token = d.b_token; a.c_batch = d.c_batch; a.c_token = d.c_token;
  return a;
}

// Few rows leave CUs idle: with at most one row per CU the sequence is cut
// into segments, up to three workgroups per CU (what the scan's registers
// allow; the state walk's allow four at N <= 64), of at least two chunks each.
// Measured, us of the call at targets of two, three and four per CU: 65536
// tokens of 24 heads of 64, N 64: 332, 304 and 318; 2 x 2048 tokens of 24 heads
// of 64, N 128: 57, 54 and 54; 3 x 777 tokens of 10 fp32 heads of 40, N 24: 31
// each (42 with segments of at least four chunks).
void heads_segments(int64_t rows, int64_t L, int64_t unit, int64_t* nseg, int64_t* seg_len) {
  *nseg = 1;
  *seg_len = L;
  const int64_t cus = cu_count();
  if (rows <= 0 || rows > cus) return;
  int64_t s = 3 * cus / rows;
  const int64_t most = L / (2 * kHQ);
  if (s > most) s = most;
  if (s <= 1) return;
  const int64_t len = ((L + s - 1) / s + unit - 1) / unit * unit;
  *nseg = (L + len - 1) / len;
  *seg_len = *nseg > 1 ? len : L;
}

}  // namespace s6i

using namespace s6i;

extern "C" {

int s6_heads_scan_fwd_workspace_size(const s6_heads_dims* d, int in_dtype, size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  const int rc = check_heads(d, in_dtype, 0, false, false, true);
  if (rc) return rc;
  *bytes = 0;
  if (d->batch == 0 || d->heads == 0 || d->seqlen == 0) return S6_OK;
  *bytes = fwd_ws(*d, heads_plan(*d, in_dtype, nullptr, nullptr, nullptr, nullptr)).total;
  return S6_OK;
}

int s6_heads_scan_fwd(const s6_heads_dims* d, int in_dtype, int flags, const void* x, const void* delta,
                      const float* delta_bias, const float* A, const void* Bm, const void* Cm, const float* D,
                      const float* h0, void* y, float* h_last, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_heads(d, in_dtype, flags, delta != nullptr, delta_bias != nullptr, true);
  if (rc) return rc;
  if (d->batch == 0 || d->heads == 0) return S6_OK;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4;
  if (d->seqlen > 0 && (!x || !A || !Bm || !Cm || !y)) return S6_ERR_NULL;
  const void* ins[] = {x, delta, Bm, Cm, y};
  for (const void* p : ins)
    if (!aligned(p, esz)) return S6_ERR_ALIGN;
  const void* f32s[] = {delta_bias, A, D, h0, h_last};
  for (const void* p : f32s)
    if (!aligned(p, 4)) return S6_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (d->seqlen == 0)
    return h_last ? launch_copy_state(h0, h_last, d->batch * d->heads * d->headdim * d->dstate, st) : S6_OK;
  HeadsPlan p = heads_plan(*d, in_dtype, x, Bm, Cm, nullptr);
  // y is stored four channels at a time
  p.vec = p.vec && aligned(y, 4 * esz);
  const FwdWs ws = fwd_ws(*d, p);
  if (ws.total > 0) {
    if (!workspace || workspace_bytes < ws.total) return S6_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return S6_ERR_ALIGN;
  }
  HeadsArgs a = heads_args(*d, p, flags, x, delta, delta_bias, A, Bm, Cm, D, h0);
  a.y = y; a.h_last = h_last; a.nseg = ws.nseg; a.seg_len = ws.seg_len;
  if (ws.nseg > 1) {
    char* w = static_cast<char*>(workspace);
    a.agg = reinterpret_cast<float*>(w + ws.agg);
    a.sd = reinterpret_cast<float*>(w + ws.sd);
    a.hin = reinterpret_cast<float*>(w + ws.hin);
    rc = launch_heads_state(in_dtype, a, p, 0, 1, st);
    if (rc == S6_OK) rc = launch_heads_fold(a, p, 1, st);
    if (rc) return rc;
  }
  return in_dtype == S6_BF16 ? launch_scan_in<uint16_t>(a, p, st) : launch_scan_in<float>(a, p, st);
}

}  // extern "C"
