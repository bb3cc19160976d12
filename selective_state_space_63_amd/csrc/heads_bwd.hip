// heads_bwd.hip -- gradients of the multi-head scan (s6_heads_scan_bwd).
//
// With the adjoint L_t = dy_t C_t^T + e^{a_{t+1}} L_{t+1} of the state (a_t =
// s_t A):
//   dx_t = w_t L_t B_t + D dy_t     dB_t = sum over heads of w_t L_t^T x_t
//   dC_t = sum over heads of S_t^T dy_t             dw_t = x_t . L_t B_t
//   G_t = <L_t, e^{a_t} S_{t-1}>    (gradient of a_t)
//   ds_t = A G_t + dw_t,  dA = sum s_t G_t,  dD = sum x_t . dy_t
// In a block of Q tokens, S entering it and L entering it from its end, with
// c the running sum of the log decays, E_ts = (dy_t . x_s)(C_t . B_s) e^{c_t - c_s}:
//   dx_s = sum_{t>=s} (C_t . B_s) e^{c_t - c_s} w_s dy_t + w_s e^{c_Q - c_s} L B_s + D dy_s
//   dC_t = sum_s P_ts B_s + e^{c_t} S^T dy_t,   P_ts = (dy_t . x_s) e^{c_t - c_s} w_s
//   dB_s = sum_t P_ts C_t + w_s e^{c_Q - c_s} L^T x_s
//   G_t  = sum_{u >= t > s} w_s E_us                      (both inside)
//        + sum_{u >= t} e^{c_u} dy_u . S C_u              (from before the block)
//        + sum_{s < t} w_s e^{c_Q - c_s} x_s . L B_s      (to after the block)
//        + e^{c_Q} <L, S>                                 (through it)
// Where a decay is strong G_t is far smaller than what lies on either side of
// t, so no part of it is taken as a difference of running totals: the sums over
// u >= t and over s < t run from their own ends, and the part inside the block
// is added up from 16 x 16 tiles of w E with t in tile T: the tiles with rows
// after T and columns before T, the rows from t on of the tiles left of (T, T),
// the columns before t of the tiles below it, and the corner of (T, T) itself.
// (From totals and prefixes, a fp32 head with A = -20 and steps of 1 missed dA by
// 4e-3 of its terms, and a reset's step added rounding noise times itself.)
//
// Two phases.  s6_heads_state_kernel walks the sequence in both directions
// and stores S and L entering every block (fp32, in operand order).  Then a workgroup of eight waves owns one block of one
// sequence and a run of a group's heads: B, C, their Gram matrix and the
// sums over heads -- dB, dC and P -- stay on chip while it goes through the
// heads, so x, dy and the states are read once and dx is written once.  The
// block is Q = 128 tokens for bf16 (64 for fp32, whose tiles are twice the
// size): the states are 8 bytes per state element and block against 6 Q bytes
// per channel of x, dy and dx, and 160 KB of LDS hold no more.
//
// Waves: wave w owns the 16 state columns n of strip w % NS in the products
// with S and L (dC, dB: rows n, columns t), all of them in registers, and
// for dx the channel tile w % 4 of every second token tile.  Wave 7 forms the
// next head's decays, waves 4 and 5 finish the last head's step gradients
// behind the next turn's barrier, so neither is waited for.
//
// Roundings (bf16 inputs): the decayed Gram matrix, P and, for dx, L enter products
// as two bf16 parts (within 2^-17), so that dx, dB and dC meet one rounding, their
// own.  The step's and the decay's gradients come from fp32 products and from S and
// L in full (three bf16 parts): two left 2e-6 to 3e-6 in dA, where fp32 sums leave
// 3e-7, and take the block kernel 494 us instead of 524 (8 x 2048 tokens of 80
// heads of 64, N 128).
//
// What bounds it: one workgroup of eight waves fits a CU (242 VGPRs, 159 KB of
// LDS), so a turn is the sum of its phases' latencies: 13 us at 128 tokens x 64
// channels x N 128.  8 x 2048 tokens of 80 heads of 64, N 128: 522 - 555 us, of
// which HBM needs 190 (1.2 GB); vector units 50 %, matrix units 17 %, LDS 31 %
// busy (31 % of that bank conflicts), half of the waves' cycles are waits.  Of it
// the second parts for dx, with their two barriers, are 43 us.  Register spills
// cost the most on the way here (802 us with 163 of them): reloads wait behind the
// prefetches of the next turn, so those are L2 touches for the states, and token
// tiles past the sequence are left out by branches.
#include "heads_kernel.h"

namespace s6i {

namespace {

template <typename In>
constexpr int kBQ = sizeof(In) == 2 ? 128 : 64;  // tokens per block (kBlockTokens of heads_state.hip)

struct HeadsBwdArgs {
  HeadsArgs h;
  void* dx;
  void* ddelta;           // or null
  void* dB;
  void* dC;
  float* parts;           // (3, batch * nblk * Q / 64, heads): dA, dD, dbias per 64 tokens
  float* bc;              // (nhb, 2, batch * L, groups, NT) partial dB, dC, or null (one head run)
  int64_t nblk, rows;
  uint32_t id0;           // first workgroup of this launch
  int groups, nhb, hpb;   // head runs of a group and heads per run
  int want_d;
};

// Offsets in LDS (bytes).
template <typename In, int NT>
struct BwdLds {
  static constexpr int Q = kBQ<In>;
  static constexpr int NTT = Q / 16, H = NTT / 2, NTILE = NTT * (NTT + 1) / 2;
  static constexpr int NFRAG = H * (H + 1);
  using XT = RowTile<In, kTP>;   // x, dy: by tokens
  using BT = RowTile<In, NT>;    // B, C: by tokens
  using LT = ColTile<In, kTP>;   // L: by states, read down its columns
  using PT = RowTile<In, Q>;     // P at the end, in the place of x and dy
  static constexpr int NS = NT / 16;
  static constexpr int bs = 0;
  static constexpr int cm = bs + BT::size(Q) * (int)sizeof(In);
  static constexpr int xs = cm + BT::size(Q) * (int)sizeof(In);
  static constexpr int ys = xs + XT::size(Q) * (int)sizeof(In);
  static constexpr int lm = ys + XT::size(Q) * (int)sizeof(In);
  static constexpr int mf = lm + LT::size(NT) * (int)sizeof(In);
  static constexpr int rp = mf + NFRAG * 512 * (int)sizeof(In);  // row sums by column tile (token, tile)
  static constexpr int cp = rp + Q * NTT * 4;                    // column sums by row tile (token, tile)
  static constexpr int yp = cp + Q * NTT * 4;                    // dy . S C by strip (token, strip)
  static constexpr int up = yp + NS * Q * 4;                     // x . L B by strip (token, strip)
  static constexpr int tok = up + NS * Q * 4;                    // per-token values, three turns' worth
  static constexpr int th = tok + 3 * 7 * Q * 4;                 // <L, S> by strip
  static constexpr int dd = th + 8 * 4;                          // x . dy by diagonal tile
  static constexpr int tb = dd + 8 * 4;                          // by token tile, see finish()
  static constexpr int total = tb + (2 * NTT + NTT * NTT) * 4;
  static_assert(total <= 163840, "LDS");
};

// First operand of the decayed Gram matrix's column tile J, in units of 512
// elements: the token pairs kk = J/2 .. H - 1 follow.
template <int H>
__device__ __forceinline__ int frag_at(int J, int kk) {
  const int m = J >> 1;
  return 2 * m * H - m * (m - 1) + ((J & 1) ? H - m : 0) + kk - m;
}

template <typename In, int NT, bool VEC>
__global__ __launch_bounds__(512) void s6_heads_bwd_kernel(HeadsBwdArgs ba) {
  using O = BwdLds<In, NT>;
  constexpr int Q = O::Q, NTT = O::NTT, H = O::H, NS = O::NS, NK = NT / 32;
  constexpr int TPN = 8 / NS, TT = NTT / TPN;       // token parts of the strips, tiles per part
  constexpr int SLOTS = (O::NTILE + 7) / 8;         // Gram tiles per wave
  constexpr int PL = Q / 64;                        // tokens per lane of a wave
  extern __shared__ __align__(16) char lds[];
  const typename O::BT bs{reinterpret_cast<In*>(lds + O::bs)}, cm{reinterpret_cast<In*>(lds + O::cm)};
  const typename O::XT xs{reinterpret_cast<In*>(lds + O::xs)}, ys{reinterpret_cast<In*>(lds + O::ys)};
  const typename O::LT lm{reinterpret_cast<In*>(lds + O::lm)};
  In* mf = reinterpret_cast<In*>(lds + O::mf);
  float* rp = reinterpret_cast<float*>(lds + O::rp);
  float* cp = reinterpret_cast<float*>(lds + O::cp);
  float* yp = reinterpret_cast<float*>(lds + O::yp);
  float* up = reinterpret_cast<float*>(lds + O::up);
  float* tok = reinterpret_cast<float*>(lds + O::tok);
  float* th = reinterpret_cast<float*>(lds + O::th);
  float* ddp = reinterpret_cast<float*>(lds + O::dd);
  float* const tb_y = reinterpret_cast<float*>(lds + O::tb);  // dy . S C of a token tile
  float* const tb_u = tb_y + NTT;                             // w x . L B of a token tile
  float* const tb_in = tb_u + NTT;                            // (j, T): w E, rows of tile T, columns before tile j

  const HeadsArgs& a = ba.h;
  uint32_t id = ba.id0 + blockIdx.x;  // (sequence, group, head run, block), the block fastest; below 2^31
  const uint32_t nb = (uint32_t)ba.nblk;
  const int64_t blk = __builtin_amdgcn_readfirstlane(id % nb);
  id /= nb;
  const int hb = __builtin_amdgcn_readfirstlane(id % (uint32_t)ba.nhb);
  id /= (uint32_t)ba.nhb;
  const int grp = __builtin_amdgcn_readfirstlane(id % (uint32_t)ba.groups);
  const int64_t b = __builtin_amdgcn_readfirstlane(id / (uint32_t)ba.groups);
  const int lane0 = threadIdx.x & 63, wv = wave_index(), g0 = lane0 >> 4, c0 = lane0 & 15;
  int lane = lane0, g = g0, c = c0;
  const int ns = wv % NS, tp = TPN == 1 ? 0 : wv / NS;
  const int64_t t0 = blk * Q;
  const int rows = (int)(a.L - t0 < Q ? a.L - t0 : Q);
  const int64_t hp = (int64_t)a.heads * a.headdim;
  const int hd0 = grp * a.hpg + hb * ba.hpb;
  const int hd1 = hb * ba.hpb + ba.hpb < a.hpg ? hd0 + ba.hpb : (grp + 1) * a.hpg;

  {
    TileRegs<In, Q, NT, 512, VEC> br, cr;
    br.load(static_cast<const In*>(a.Bm) + b * a.b_batch + t0 * a.b_token + (int64_t)grp * a.dstate, a.b_token, rows,
            a.dstate);
    cr.load(static_cast<const In*>(a.Cm) + b * a.c_batch + t0 * a.c_token + (int64_t)grp * a.dstate, a.c_token, rows,
            a.dstate);
    br.mask(rows, a.dstate);
    cr.mask(rows, a.dstate);
    br.store(bs);
    cr.store(cm);
  }
  // what lies above the diagonal stays 0
  for (int i = threadIdx.x; i < O::NFRAG * 512; i += 512) mf[i] = In(0);
  for (int i = threadIdx.x; i < Q * NTT; i += 512) rp[i] = cp[i] = 0.0f;
  // and what lies past the sequence: its token tiles are left out below
  for (int i = threadIdx.x; i < Q * NS; i += 512) yp[i] = up[i] = 0.0f;
  if (threadIdx.x < 8) ddp[threadIdx.x] = 0.0f;
  if (threadIdx.x < NTT * NTT) tb_in[threadIdx.x] = 0.0f;

  TileRegs<In, Q, kTP, 512, VEC> xr, yr;
  auto issue = [&](int hd, int pt) {
    const int on = hd < hd1 ? rows : 0, cols = a.headdim - pt * kTP;
    const int64_t col = (int64_t)hd * a.headdim + pt * kTP;
    xr.load(static_cast<const In*>(a.x) + b * a.x_batch + t0 * a.x_token + col, a.x_token, on, cols < kTP ? cols : kTP);
    yr.load(static_cast<const In*>(a.dy) + (b * a.L + t0) * hp + col, hp, on, cols < kTP ? cols : kTP);
  };
  // The last wave forms a head's per-token values a turn ahead, from steps
  // loaded another turn earlier and kept as loaded: running log2 decay (its
  // second part is the last value), its exponential, input weight, decay to the
  // block's end, step, and the step's derivative.
  In draw[PL];
  auto issue_step = [&](int hd) {
    if (wv != 7 || hd >= hd1 || !a.delta) return;
#pragma unroll
    for (int k = 0; k < PL; ++k)
      load_step<In, VEC>(draw[k], static_cast<const In*>(a.delta) + b * a.d_batch + (t0 + k * 64) * a.d_token + hd,
                         a.d_token, lane, rows - k * 64);
  };
  // the head of the turn after (hd, pt)
  auto after = [&](int hd, int pt) { return pt + 1 == a.ptiles ? hd + 1 : hd; };
  auto decays = [&](int hd, int buf) {
    if (wv != 7 || hd >= hd1) return;
    const float bias = a.dbias ? a.dbias[hd] : 0.0f, a2 = a.A[hd] * kLog2e;
    float* o = tok + buf * 7 * Q;
    LogSum base = {0.0f, 0.0f}, cl[PL];
#pragma unroll
    for (int k = 0; k < PL; ++k) {
      const int t = k * 64 + lane;
      const bool on = t < rows;
      const float v = to_f32(draw[k]) + bias;
      const float sv = on ? step_of(a, to_f32(draw[k]), bias) : 0.0f;
      const LogSum sum = log_scan(on ? clamp_log2(sv * a2) : 0.0f);
      cl[k] = {base.hi + sum.hi, base.lo + sum.lo};
      base = last_lane(cl[k]);
      o[t] = cl[k].hi;
      o[6 * Q + t] = cl[k].lo;
      o[Q + t] = fast_exp2(cl[k].hi + cl[k].lo);
      o[2 * Q + t] = on ? (a.unit ? 1.0f : sv) : 0.0f;
      o[4 * Q + t] = sv;
      o[5 * Q + t] = a.softplus ? fast_rcp(1.0f + fast_exp2(-v * kLog2e)) : 1.0f;
    }
#pragma unroll
    for (int k = 0; k < PL; ++k) o[3 * Q + k * 64 + lane] = decay_between(base, cl[k]);
  };
#pragma unroll
  for (int k = 0; k < PL; ++k) draw[k] = In(0);
  issue_step(hd0);
  issue(hd0, 0);
  decays(hd0, 0);
  issue_step(after(hd0, 0));
  __syncthreads();

  // Gram tiles of this wave (rows t of tile I, columns s of tile J <= I)
  const int b_row = O::BT::row_lane(g, c);
  int tI[SLOTS], tJ[SLOTS];
  f32x4 CB[SLOTS], P[SLOTS];
#pragma unroll
  for (int k = 0; k < SLOTS; ++k) {
    const int n = 8 * k + wv;
    int I = 0;
#pragma unroll
    for (int i = 1; i < NTT; ++i) I += n >= i * (i + 1) / 2 ? 1 : 0;
    tI[k] = I;
    tJ[k] = n - I * (I + 1) / 2;
    CB[k] = P[k] = f32x4{0, 0, 0, 0};
    if (n < O::NTILE) {
#pragma unroll
      for (int kk = 0; kk < NK; ++kk)
        CB[k] = mma(cm.row(b_row, 16 * I, kk), bs.row(b_row, 16 * tJ[k], kk), CB[k]);
    }
  }
  f32x4 dC[TT], dB[TT];
#pragma unroll
  for (int i = 0; i < TT; ++i) dC[i] = dB[i] = f32x4{0, 0, 0, 0};

  float acc_g = 0.0f, acc_ds = 0.0f, acc_d = 0.0f;  // sums over the channel tiles of a head

  // dx of a turn is stored in the next one, behind the wait for its inputs
  // (stores before it would be waited for as well)
  Four<In> dxv[NTT / 2];
  const uint32_t x_row = (uint32_t)hp * (uint32_t)sizeof(In);
  auto put_dx = [&](int hd, int pt) {
    const int p = 16 * (wv & 3) + 4 * g, pleft = a.headdim - pt * kTP;
    In* const base = static_cast<In*>(ba.dx) + (b * a.L + t0) * hp + (int64_t)hd * a.headdim + pt * kTP;
    if constexpr (VEC) {  // rows past the sequence and channels past the head are dropped
      const __amdgpu_buffer_rsrc_t db =
          buffer_of(base, (uint32_t)(rows - 1) * x_row + (uint32_t)(pleft < kTP ? pleft : kTP) * (uint32_t)sizeof(In));
      const uint32_t off = (uint32_t)(16 * (wv >> 2) + c) * x_row + (uint32_t)p * (uint32_t)sizeof(In);
#pragma unroll
      for (int i = 0; i < NTT / 2; ++i) dxv[i].store(db, p < pleft ? off + (uint32_t)(32 * i) * x_row : kNowhere);
    } else {
#pragma unroll
      for (int i = 0; i < NTT / 2; ++i) {
        const int s = 16 * (2 * i + (wv >> 2)) + c;
        if (s < rows) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (p + r < pleft) base[s * hp + p + r] = dxv[i].get(r);
        }
      }
    }
  };
  // A head's stored states (S; L lies nblk rows tiles behind).  touch() reads
  // one word of each of their cache lines a turn ahead, so that they come from
  // L2 when the operands are loaded: held in registers from there on, they
  // would not leave room for the sums.
  constexpr int64_t kTile = (int64_t)kTP * NT;
  auto state_at = [&](int hd, int pt) {
    const int64_t row = (b * a.heads + hd) * (int64_t)a.ptiles + pt;
    return a.planes + (blk * ba.rows + row) * kTile;
  };
  uint32_t touched = 0;
  auto touch = [&](int hd, int pt) {
    constexpr int kLines = (int)(kTile * sizeof(float) / 128);
    static_assert(kLines <= 256, "one line of S and L per thread");
    if (hd < hd1 && (threadIdx.x & 255) < kLines) {
      const float* sp = state_at(hd, pt) + (threadIdx.x >> 8) * (ba.nblk * ba.rows * kTile);
      touched = reinterpret_cast<const uint32_t*>(sp)[(threadIdx.x & 255) * 32];
    }
  };
  // Waves 4 and 5 (fp32: 4), 64 tokens each, for the turn before: the decay's and
  // the step's gradients.  What a token needs of the other tiles of tokens is
  // left in LDS by tile (tb_*).
  const bool tokens_wave = wv >= 4 && wv < 4 + PL;
  float e_in = 0.0f, e_row = 0.0f, e_col = 0.0f, e_y = 0.0f, e_u = 0.0f, e_w = 0.0f, through = 0.0f;
  int done_hd = -1, done_buf = 0;
  bool done_last = false;
  auto finish = [&]() {
    if (!tokens_wave || done_hd < 0) return;
    const float Ah = a.A[done_hd];
    const int T = 4 * (wv - 4) + (lane >> 4);
    float in = e_in + row_from(e_row) + row_before(e_col), y = row_from(e_y), u = row_before(e_u);
    float v[3][NTT];
#pragma unroll
    for (int j = 0; j < NTT; j += 4) {
      *reinterpret_cast<float4*>(&v[0][j]) = *reinterpret_cast<const float4*>(tb_in + T * NTT + j);
      *reinterpret_cast<float4*>(&v[1][j]) = *reinterpret_cast<const float4*>(tb_y + j);
      *reinterpret_cast<float4*>(&v[2][j]) = *reinterpret_cast<const float4*>(tb_u + j);
    }
#pragma unroll
    for (int j = 0; j < NTT; ++j) {
      in += v[0][j];
      y += j > T ? v[1][j] : 0.0f;
      u += j < T ? v[2][j] : 0.0f;
    }
    const float* o = tok + done_buf * 7 * Q;
    const int t = 64 * (wv - 4) + lane;
    // A decay taken as 0 (see clamp_log2) has no gradient, and the products of its
    // step and A, either of which may be infinite, with 0 are left out.
    const float step = o[4 * Q + t];
    const bool gone = step * (Ah * kLog2e) <= kMinLog2;
    const float G = gone ? 0.0f : (in + u) + (y + through);
    acc_g += G;
    acc_ds = (gone ? acc_ds : __builtin_fmaf(Ah, G, acc_ds)) + (a.unit ? 0.0f : e_w);
    if (!done_last) return;
    const float dv = acc_ds * o[5 * Q + t];
    if (t < rows && ba.ddelta)
      static_cast<In*>(ba.ddelta)[(b * a.L + t0 + t) * a.heads + done_hd] = from_f32<In>(dv);
    const float sa = wave_sum(t < rows && !gone ? step * acc_g : 0.0f), sb = wave_sum(t < rows ? dv : 0.0f);
    if (lane == 0) {
      const int64_t n = a.batch * ba.nblk * PL, at = ((b * ba.nblk + blk) * PL + (wv - 4)) * a.heads + done_hd;
      ba.parts[at] = sa;
      ba.parts[n * a.heads + at] = acc_d;
      ba.parts[2 * n * a.heads + at] = sb;
    }
    acc_g = acc_ds = acc_d = 0.0f;
  };
  int buf = 0;
  auto next = [](int i) { return i == 2 ? 0 : i + 1; };
  for (int hd = hd0; hd < hd1; ++hd) {
    const float dsk = a.D ? a.D[hd] : 0.0f;
    for (int pt = 0; pt < a.ptiles; ++pt, buf = next(buf)) {
      const bool last_pt = pt + 1 == a.ptiles;
      // LDS addresses are formed again in every turn: kept across it they
      // would not leave room for the sums
      lane = lane0;
      asm volatile("" : "+v"(lane));
      g = lane >> 4; c = lane & 15;
      const int x_row = O::XT::row_lane(g, c), b_row = O::BT::row_lane(g, c);
      const int p0 = pt * kTP, pleft = a.headdim - p0;
      asm volatile("" ::"v"(touched));
      xr.mask(rows, pleft < kTP ? pleft : kTP);
      yr.mask(rows, pleft < kTP ? pleft : kTP);
      xr.store(xs);
      yr.store(ys);
      decays(after(hd, pt), next(buf));
      if (hd > hd0 || pt > 0) put_dx(pt > 0 ? hd : hd - 1, pt > 0 ? pt - 1 : a.ptiles - 1);
      const float* cs = tok + buf * 7 * Q;
      const float *ec = cs + Q, *ww = cs + 2 * Q, *wd = cs + 3 * Q, *cl = cs + 6 * Q;
      __syncthreads();
      finish();
      issue_step(last_pt ? after(hd + 1, 0) : after(hd, pt + 1));
      touch(after(hd, pt), last_pt ? 0 : pt + 1);

      // the decays of Gram tile (I, J) of this wave
      auto tile_decays = [&](int I, int J, float (&l)[4]) {
        const float4 ct4 = *reinterpret_cast<const float4*>(cs + 16 * I + 4 * g);
        const float4 lt4 = *reinterpret_cast<const float4*>(cl + 16 * I + 4 * g);
        const float ct[4] = {ct4.x, ct4.y, ct4.z, ct4.w}, lt[4] = {lt4.x, lt4.y, lt4.z, lt4.w};
        const float cj = cs[16 * J + c], lj = cl[16 * J + c];
#pragma unroll
        for (int r = 0; r < 4; ++r) l[r] = decay_between(ct[r], lt[r], cj, lj);
      };
      // inside the block
      Frag<float> Sf[2], Lf[2];
      Four<In> m_lo[SLOTS];  // second parts of the decayed Gram tiles
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) {
        if (k == SLOTS - 1) {
          // states entering the block: this wave's strip of n, all 64 channels
          // (touched a turn ago: they come from L2)
          const float* sp = state_at(hd, pt) + ns * 1024;
          const float* lp = sp + ba.nblk * ba.rows * kTile;
          const uint32_t off = (uint32_t)lane * 16;
#pragma unroll
          for (int pp = 0; pp < 2; ++pp) {
            load_halves(scalar_base(sp + pp * 512) + off, Sf[pp]);
            load_halves(scalar_base(lp + pp * 512) + off, Lf[pp]);
          }
        }
        const int n = 8 * k + wv;
        if (n < O::NTILE && 16 * tI[k] < rows) {
          const int I = tI[k], J = tJ[k];
          f32x4 X = {0, 0, 0, 0};
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            X = mma(ys.row(x_row, 16 * I, kk), xs.row(x_row, 16 * J, kk), X);
          const float wj = ww[16 * J + c];
          float l[4], m[4], er[4], col = 0.0f, diag = 0.0f;
          tile_decays(I, J, l);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const bool on = I != J || 4 * g + r >= c;
            const float m0 = on ? CB[k][r] * l[r] : 0.0f;
            const float e0 = on ? m0 * X[r] : 0.0f;
            m[r] = m0 * wj;
            er[r] = e0 * wj;
            col += e0;
            P[k][r] += on ? X[r] * (l[r] * wj) : 0.0f;
            if (I == J && 4 * g + r == c) diag = X[r];
          }
          In* const at = mf + frag_at<H>(J, I >> 1) * 512 + lane * 8 + 4 * (I & 1);
          if constexpr (sizeof(In) == 2) {
            Four<In> hi;
            hi.split(m);
            hi.put(at);
            m_lo[k].set(m);
          } else {
            store_vec<In, 4>(at, m);
          }
          if (I == J) corner(er, g, c);  // a row's own part of G, in the place of its sum
#pragma unroll
          for (int r = 0; r < 4; ++r) er[r] = row_sum(er[r]);
          // (every lane of a sum writes it: the same value to the same place)
#pragma unroll
          for (int r = 0; r < 4; ++r) rp[(16 * I + 4 * g + r) * NTT + J] = er[r];
          cp[(16 * J + c) * NTT + I] = half_sum(pair_row_sum(col));
          if (I == J && ba.want_d) ddp[I] = wave_sum(diag);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (tp == 0) {
        float s = 0.0f;
#pragma unroll
        for (int pp = 0; pp < 2; ++pp)
#pragma unroll
          for (int e = 0; e < 8; ++e) s = __builtin_fmaf(Sf[pp].v[e], Lf[pp].v[e], s);
        th[ns] = wave_sum(s);
      }
      // from before the block
      {
        Whole<In> sw[2];
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) to_whole(Sf[pp].v, sw[pp]);
#pragma unroll
        for (int i = 0; i < TT; ++i) {
          const int t = 16 * (tp * TT + i) + c;
          if (t - c >= rows) continue;
          f32x4 U = {0, 0, 0, 0};
#pragma unroll
          for (int pp = 0; pp < 2; ++pp) U = mma_whole(sw[pp], ys.row(x_row, t - c, pp), U);
          float cv[4], sy = 0.0f;
          cm.four(t, 4 * ns + g, cv);
          const float e = ec[t];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            sy = __builtin_fmaf(cv[r], U[r], sy);
            dC[i][r] = __builtin_fmaf(e, U[r], dC[i][r]);
          }
          yp[t * NS + ns] = e * half_sum(pair_row_sum(sy));
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      // to after the block
      Whole<In> lw[2];
#pragma unroll
      for (int pp = 0; pp < 2; ++pp) to_whole(Lf[pp].v, lw[pp]);
#pragma unroll
      for (int i = 0; i < TT; ++i) {
        const int t = 16 * (tp * TT + i) + c;
        if (t - c >= rows) continue;
        f32x4 V = {0, 0, 0, 0};
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) V = mma_whole(lw[pp], xs.row(x_row, t - c, pp), V);
        float bv[4], su = 0.0f;
        bs.four(t, 4 * ns + g, bv);
        const float f = wd[t], fw = ww[t] * f;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          su = __builtin_fmaf(bv[r], V[r], su);
          dB[i][r] = __builtin_fmaf(fw, V[r], dB[i][r]);
        }
        up[t * NS + ns] = f * half_sum(pair_row_sum(su));
        __builtin_amdgcn_sched_barrier(0);
      }

      // a part of L by states, this wave's strip
      auto put_l = [&](const typename O::LT& to, int part) {
        if (tp != 0) return;
#pragma unroll
        for (int pp = 0; pp < 2; ++pp) {
          float f[4], h[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[e] = frag_f32(lw[pp].part[part], e);
            h[e] = frag_f32(lw[pp].part[part], 4 + e);
          }
          store_vec<In, 4>(to.t + to.at(16 * ns + c, 8 * pp + g), f);
          store_vec<In, 4>(to.t + to.at(16 * ns + c, 8 * pp + 4 + g), h);
        }
      };
      put_l(lm, 0);
      __syncthreads();
      issue(after(hd, pt), last_pt ? 0 : pt + 1);

      // dx, transposed: channels of tile q, tokens of tiles J.  bf16: the second
      // part of L takes the place of x, which is done, and that of the decayed Gram
      // matrix the place of the first, once that is.
      {
        const int q = wv & 3;
        const auto l_col = O::LT::col_lane(g, c);
        const typename O::LT ll{xs.t};
        f32x4 acc[NTT / 2];
        Frag<In> yq[H];
        auto inside = [&]() {  // acc += dy^T M, for the part of M that is there
#pragma unroll
          for (int i = 0; i < NTT / 2; ++i) {
            const int J = 2 * i + (wv >> 2);
            if (16 * J >= rows) continue;
#pragma unroll
            for (int kk = i; kk < H; ++kk) acc[i] = mma(yq[kk], lane_frag(mf + frag_at<H>(J, kk) * 512, lane), acc[i]);
            __builtin_amdgcn_sched_barrier(0);
          }
        };
        if constexpr (sizeof(In) == 2) put_l(ll, 1);
#pragma unroll
        for (int kk = 0; kk < H; ++kk) yq[kk] = ys.col(q, kk, g, c);
#pragma unroll
        for (int i = 0; i < NTT / 2; ++i) {
          float dyv[4];
          ys.four(16 * (2 * i + (wv >> 2)) + c, 4 * q + g, dyv);
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][r] = dsk * dyv[r];
        }
        inside();
        if constexpr (sizeof(In) == 2) {
          __syncthreads();
#pragma unroll
          for (int k = 0; k < SLOTS; ++k)
            if (8 * k + wv < O::NTILE && 16 * tI[k] < rows)
              m_lo[k].put(mf + frag_at<H>(tJ[k], tI[k] >> 1) * 512 + lane * 8 + 4 * (tI[k] & 1));
        }
        f32x4 lb[NTT / 2];  // B L, from after the block
#pragma unroll
        for (int i = 0; i < NTT / 2; ++i) lb[i] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int kk = 0; kk < NK; ++kk) {
          Pair<In> lq;
          lq.hi = lm.col(l_col, q, kk, g, c);
          if constexpr (sizeof(In) == 2) lq.lo = ll.col(l_col, q, kk, g, c);
#pragma unroll
          for (int i = 0; i < NTT / 2; ++i) lb[i] = mma_pair(lq, bs.row(b_row, 16 * (2 * i + (wv >> 2)), kk), lb[i]);
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < NTT / 2; ++i) {
          const int s = 16 * (2 * i + (wv >> 2)) + c;
          acc[i] += lb[i] * (ww[s] * wd[s]);
        }
        if constexpr (sizeof(In) == 2) {
          __syncthreads();
          inside();
        }
#pragma unroll
        for (int i = 0; i < NTT / 2; ++i) {
          const float o[4] = {acc[i][0], acc[i][1], acc[i][2], acc[i][3]};
          dxv[i].set(o);
        }
      }
      __syncthreads();

      // Waves 4 and 5 take the sums over tiles and strips now (they are written
      // again after the next barrier) and finish them behind that barrier.  A
      // row's sums right of its tile and a column's above it are 0.
      if (tokens_wave) {
        const int t = 64 * (wv - 4) + lane, T = t >> 4;
        float v[2][NTT];
#pragma unroll
        for (int j = 0; j < NTT; j += 4) {
          *reinterpret_cast<float4*>(&v[0][j]) = *reinterpret_cast<const float4*>(rp + t * NTT + j);
          *reinterpret_cast<float4*>(&v[1][j]) = *reinterpret_cast<const float4*>(cp + t * NTT + j);
        }
        float R = 0.0f, K = 0.0f, own = 0.0f;
#pragma unroll
        for (int j = 0; j < NTT; ++j) {
          // the rows of tile T, columns before tile j < T
          if (j > 0 && j < NTT - 1) tb_in[j * NTT + T] = row_sum(j < T ? R : 0.0f);
          R += j < T ? v[0][j] : 0.0f;
          K += j > T ? v[1][j] : 0.0f;
          e_in = j == T ? v[0][j] : e_in;
          own = j == T ? v[1][j] : own;
        }
        float w[2][NS], Y = 0.0f, U = 0.0f;
#pragma unroll
        for (int j = 0; j < NS; j += 2) {
          *reinterpret_cast<float2*>(&w[0][j]) = *reinterpret_cast<const float2*>(yp + t * NS + j);
          *reinterpret_cast<float2*>(&w[1][j]) = *reinterpret_cast<const float2*>(up + t * NS + j);
        }
#pragma unroll
        for (int j = 0; j < NS; ++j) { Y += w[0][j]; U += w[1][j]; }
        const float wt = ww[t];
        e_row = R;
        e_col = wt * K;
        e_y = Y;
        e_u = wt * U;
        e_w = (K + own) + U;
        tb_y[T] = row_sum(e_y);
        tb_u[T] = row_sum(e_u);
        through = 0.0f;
#pragma unroll
        for (int n = 0; n < NS; ++n) through += th[n];
        through *= ec[Q - 1];
        if (ba.want_d && wv == 4) {
#pragma unroll
          for (int I = 0; I < NTT; ++I) acc_d += ddp[I];
        }
        done_hd = hd;
        done_last = last_pt;
        done_buf = buf;
      }
    }
  }

  __syncthreads();
  finish();
  put_dx(hd1 - 1, a.ptiles - 1);

  // dC += P B and dB += P^T C with P summed over the heads.  Every wave is past
  // the last barrier, so all but the tokens' values is free: P lies in the place of
  // x and dy, its second bf16 part in that of L and the decayed Gram matrix.
  {
    const typename O::PT pm{xs.t}, pl{lm.t};
    static_assert(O::PT::size(Q) <= 2 * O::XT::size(Q), "P fits x and dy");
    static_assert(sizeof(In) == 4 || O::PT::size(Q) * 2 <= O::tok - O::lm, "and its second part");
    auto put = [&](int at, float v) {
      pm.t[at] = from_f32<In>(v);
      if constexpr (sizeof(In) == 2) pl.t[at] = from_f32<In>(v - (float)(__bf16)v);
    };
#pragma unroll
    for (int k = 0; k < SLOTS; ++k) {
      if (8 * k + wv < O::NTILE) {
#pragma unroll
        for (int r = 0; r < 4; ++r) put(pm.at(16 * tI[k] + 4 * g + r, 4 * tJ[k] + (c >> 2)) + (c & 3), P[k][r]);
      }
    }
    if (wv < H) {  // the tile right of an even diagonal tile shares an operand with it
#pragma unroll
      for (int r = 0; r < 4; ++r) put(pm.at(32 * wv + 4 * g + r, 4 * (2 * wv + 1) + (c >> 2)) + (c & 3), 0.0f);
    }
    __syncthreads();
    const int p_row = O::PT::row_lane(g, c);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int it = tp * TT + i;
      if (16 * it >= rows) continue;
      Pair<In> p;
      for (int kk = 0; kk <= it / 2; ++kk) {
        p.hi = pm.row(p_row, 16 * it, kk);
        if constexpr (sizeof(In) == 2) p.lo = pl.row(p_row, 16 * it, kk);
        dC[i] = mma_pair(bs.col(ns, kk, g, c), p, dC[i]);
      }
      for (int kk = it / 2; kk < H; ++kk) {
        p.hi = pm.col(it, kk, g, c);
        if constexpr (sizeof(In) == 2) p.lo = pl.col(it, kk, g, c);
        dB[i] = mma_pair(cm.col(ns, kk, g, c), p, dB[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const int t = 16 * (tp * TT + i) + c, n = 16 * ns + 4 * g;
      if (t < rows) {
        const int64_t tok = b * a.L + t0 + t;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float f[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) f[r] = m ? dC[i][r] : dB[i][r];
          if (ba.bc) {
            store_vec<float, 4>(ba.bc + (((int64_t)(hb * 2 + m) * a.batch * a.L + tok) * ba.groups + grp) * NT + n, f);
          } else {
            In* o = static_cast<In*>(m ? ba.dC : ba.dB) + (tok * ba.groups + grp) * a.dstate + n;
            if constexpr (VEC) {
              if (n < a.dstate) store_vec<In, 4>(o, f);
            } else {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (n + r < a.dstate) o[r] = from_f32<In>(f[r]);
            }
          }
        }
      }
    }
  }
}

// dB, dC: the head runs' parts added in order (0 of none), four states per thread
// and turn.
template <typename In>
__global__ __launch_bounds__(256) void s6_heads_sum_bc(const float* bc, In* dB, In* dC, int64_t rows, int NT, int N,
                                                       int nhb) {
  const int per = NT / 4, m = blockIdx.y;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < rows * per; i += (int64_t)gridDim.x * 256) {
    const int64_t row = i / per;
    const int n = (int)(i - row * per) * 4;
    if (n >= N) continue;
    float s[4] = {0, 0, 0, 0};
    for (int h = 0; h < nhb; ++h) {
      float v[4];
      load_vec<float, 4>(bc + ((int64_t)(h * 2 + m) * rows + row) * NT + n, v);
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] += v[r];
    }
    In* o = (m ? dC : dB) + row * N + n;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (n + r < N) o[r] = from_f32<In>(s[r]);
  }
}

// dA, dD, dbias: the blocks' parts of one head added in a fixed order.
__global__ __launch_bounds__(256) void s6_heads_sum_parts(const float* parts, float* dA, float* dD, float* dbias,
                                                          int64_t n, int heads) {
  __shared__ float buf[4];
  const int hd = blockIdx.x, m = blockIdx.y;
  float* o = m == 0 ? dA : m == 1 ? dD : dbias;
  if (!o) return;
  float s = 0.0f;
  for (int64_t i = threadIdx.x; i < n; i += 256) s += parts[((int64_t)m * n + i) * heads + hd];
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = s;
  __syncthreads();
  if (threadIdx.x == 0) o[hd] = (buf[0] + buf[1]) + (buf[2] + buf[3]);
}

struct BwdWs {
  int64_t nblk, nseg, seg_len;
  int nhb, hpb;
  size_t planes, agg, sd, hin, parts, bc, total;
};

// Head runs of a group: one workgroup fits a CU, so a launch takes
// ceil(workgroups / CUs) rounds of a run's heads; the setup of a block and
// the parts' sums weigh about one head more per run.
void head_runs(int64_t blocks, int64_t hpg, int* nhb, int* hpb) {
  const int64_t cus = cu_count();
  double best = 0.0;
  *nhb = 1;
  *hpb = (int)hpg;
  for (int64_t n = 1; n <= hpg && n <= 64; ++n) {
    const int64_t per = (hpg + n - 1) / n, runs = (hpg + per - 1) / per;
    const double cost = (double)((blocks * runs + cus - 1) / cus) * (double)(per + 1);
    if (n == 1 || cost < best) {
      best = cost;
      *nhb = (int)runs;
      *hpb = (int)per;
    }
  }
}

BwdWs bwd_ws(const s6_heads_dims& d, const HeadsPlan& p, int in_dtype) {
  BwdWs o;
  const int64_t q = in_dtype == S6_BF16 ? kBQ<uint16_t> : kBQ<float>;
  o.nblk = (d.seqlen + q - 1) / q;
  head_runs(d.batch * d.groups * o.nblk, d.heads / d.groups, &o.nhb, &o.hpb);
  heads_segments(2 * p.rows, d.seqlen, q, &o.nseg, &o.seg_len);
  const size_t tile = (size_t)p.rows * kTP * p.NT * sizeof(float);
  o.planes = 0;
  o.agg = up256(2 * (size_t)o.nblk * tile);
  o.sd = o.agg + (o.nseg > 1 ? up256(2 * (size_t)o.nseg * tile) : 0);
  o.hin = o.sd + (o.nseg > 1 ? up256(2 * (size_t)o.nseg * p.rows * sizeof(float)) : 0);
  o.parts = o.hin + (o.nseg > 1 ? up256(2 * (size_t)o.nseg * tile) : 0);
  o.bc = o.parts + up256(3 * (size_t)d.batch * o.nblk * (q / 64) * d.heads * sizeof(float));
  o.total = o.bc + (o.nhb > 1 ? up256((size_t)o.nhb * 2 * d.batch * d.seqlen * d.groups * p.NT * sizeof(float)) : 0);
  return o;
}

template <typename In, int NT, bool VEC>
int launch_bwd_v(HeadsBwdArgs a, hipStream_t st) {
  const auto kern = s6_heads_bwd_kernel<In, NT, VEC>;
  constexpr int lds = BwdLds<In, NT>::total;
  if constexpr (lds > 65536)
    S6_HIP(hipFuncSetAttribute(reinterpret_cast<const void*>(kern), hipFuncAttributeMaxDynamicSharedMemorySize, lds),
           "s6_heads_bwd_kernel LDS size");
  const int64_t n = a.nblk * a.nhb * a.groups * a.h.batch;
  for (int64_t at = 0; at < n; at += kMaxBlocks) {
    a.id0 = (uint32_t)at;
    hipLaunchKernelGGL(kern, dim3((unsigned)(n - at < kMaxBlocks ? n - at : kMaxBlocks)), dim3(512), lds, st, a);
    S6_HIP(hipGetLastError(), "s6_heads_bwd_kernel launch");
  }
  return S6_OK;
}
template <typename In, int NT>
int launch_bwd_n(const HeadsBwdArgs& a, bool vec, hipStream_t st) {
  return vec ? launch_bwd_v<In, NT, true>(a, st) : launch_bwd_v<In, NT, false>(a, st);
}
template <typename In>
int launch_bwd_in(const HeadsBwdArgs& a, const HeadsPlan& p, bool vec, hipStream_t st) {
  if (p.NT == 32) return launch_bwd_n<In, 32>(a, vec, st);
  if (p.NT == 64) return launch_bwd_n<In, 64>(a, vec, st);
  return launch_bwd_n<In, 128>(a, vec, st);
}

template <typename In>
int launch_sum_bc(const float* bc, void* dB, void* dC, int64_t rows, int NT, int N, int nhb, hipStream_t st) {
  const int64_t n = (rows * (NT / 4) + 255) / 256;
  hipLaunchKernelGGL((s6_heads_sum_bc<In>), dim3((unsigned)(n < kMaxBlocks ? n : kMaxBlocks), 2), dim3(256), 0, st, bc,
                     static_cast<In*>(dB), static_cast<In*>(dC), rows, NT, N, nhb);
  S6_HIP(hipGetLastError(), "s6_heads_sum_bc launch");
  return S6_OK;
}

template <typename In>
int launch_sums(const HeadsBwdArgs& a, const HeadsPlan& p, float* dA, float* dD, float* dbias, hipStream_t st) {
  if (a.bc) {
    const int rc = launch_sum_bc<In>(a.bc, a.dB, a.dC, a.h.batch * a.h.L * a.groups, p.NT, a.h.dstate, a.nhb, st);
    if (rc) return rc;
  }
  hipLaunchKernelGGL(s6_heads_sum_parts, dim3((unsigned)a.h.heads, 3), dim3(256), 0, st, a.parts, dA, dD, dbias,
                     a.h.batch * a.nblk * (kBQ<In> / 64), a.h.heads);
  S6_HIP(hipGetLastError(), "s6_heads_sum_parts launch");
  return S6_OK;
}

}  // namespace

}  // namespace s6i

using namespace s6i;

extern "C" {

int s6_heads_scan_bwd_workspace_size(const s6_heads_dims* d, int in_dtype, size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  const int rc = check_heads(d, in_dtype, 0, false, false, true);
  if (rc) return rc;
  *bytes = 0;
  if (d->batch == 0 || d->heads == 0 || d->seqlen == 0) return S6_OK;
  *bytes = bwd_ws(*d, heads_plan(*d, in_dtype, nullptr, nullptr, nullptr, nullptr), in_dtype).total;
  return S6_OK;
}

int s6_heads_scan_bwd(const s6_heads_dims* d, int in_dtype, int flags, const void* x, const void* delta,
                      const float* delta_bias, const float* A, const void* Bm, const void* Cm, const float* D,
                      const float* h0, const void* dy, const float* dh_last, void* dx, void* ddelta, float* dA,
                      void* dBm, void* dCm, float* dD, float* dh0, float* ddelta_bias, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc = check_heads(d, in_dtype, flags, delta != nullptr, delta_bias != nullptr, true);
  if (rc) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t len = d->batch * d->seqlen;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4;
  const bool work = len > 0 && d->heads > 0;
  if (d->heads > 0 && !dA) return S6_ERR_NULL;
  if (work && (!x || !A || !Bm || !Cm || !dy || !dx || !dBm || !dCm || (delta && !ddelta))) return S6_ERR_NULL;
  const void* ins[] = {x, delta, Bm, Cm, dy, dx, ddelta, dBm, dCm};
  for (const void* p : ins)
    if (!aligned(p, esz)) return S6_ERR_ALIGN;
  const void* f32s[] = {delta_bias, A, D, h0, dh_last, dA, dD, dh0, ddelta_bias};
  for (const void* p : f32s)
    if (!aligned(p, 4)) return S6_ERR_ALIGN;
  if (!work) {  // empty sums
    fill(dA, 0.0f, d->heads, st);
    fill(dD, 0.0f, d->heads, st);
    fill(ddelta_bias, 0.0f, d->heads, st);
    S6_HIP(hipGetLastError(), "fill launch");
    if (len > 0 && dBm && dCm) {  // no heads
      const int n = (int)d->dstate, wide = (n + 3) / 4 * 4;
      rc = in_dtype == S6_BF16 ? launch_sum_bc<uint16_t>(nullptr, dBm, dCm, len * d->groups, wide, n, 0, st)
                               : launch_sum_bc<float>(nullptr, dBm, dCm, len * d->groups, wide, n, 0, st);
      if (rc) return rc;
    }
    return dh0 ? launch_copy_state(dh_last, dh0, d->batch * d->heads * d->headdim * d->dstate, st) : S6_OK;
  }
  const HeadsPlan p = heads_plan(*d, in_dtype, x, Bm, Cm, dy);
  const BwdWs ws = bwd_ws(*d, p, in_dtype);
  if (ws.nblk * ws.nhb * d->groups * d->batch > INT32_MAX) return S6_ERR_SHAPE;
  if (!workspace || workspace_bytes < ws.total) return S6_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return S6_ERR_ALIGN;
  char* w = static_cast<char*>(workspace);
  HeadsBwdArgs ba;
  memset(&ba, 0, sizeof(ba));
  ba.h = heads_args(*d, p, flags, x, delta, delta_bias, A, Bm, Cm, D, h0);
  HeadsArgs& a = ba.h;
  a.dy = dy; a.dh_last = dh_last; a.dh0 = dh0;
  a.nseg = ws.nseg; a.seg_len = ws.seg_len;
  if (ws.nseg > 1) {
    a.agg = reinterpret_cast<float*>(w + ws.agg);
    a.sd = reinterpret_cast<float*>(w + ws.sd);
    rc = launch_heads_state(in_dtype, a, p, 0, 2, st);
    a.hin = reinterpret_cast<float*>(w + ws.hin);
    if (rc == S6_OK) rc = launch_heads_fold(a, p, 2, st);
    if (rc) return rc;
  }
  a.planes = reinterpret_cast<float*>(w + ws.planes);
  rc = launch_heads_state(in_dtype, a, p, 1, 2, st);
  if (rc) return rc;
  ba.dx = dx; ba.ddelta = ddelta; ba.dB = dBm; ba.dC = dCm;
  ba.parts = reinterpret_cast<float*>(w + ws.parts);
  ba.bc = ws.nhb > 1 ? reinterpret_cast<float*>(w + ws.bc) : nullptr;
  ba.nblk = ws.nblk; ba.rows = p.rows; ba.groups = (int)d->groups; ba.nhb = ws.nhb; ba.hpb = ws.hpb;
  ba.want_d = dD != nullptr;
  // dx, dB and dC are stored four values at a time
  const bool vec = p.vec && aligned(dx, 4 * esz) && aligned(dBm, 4 * esz) && aligned(dCm, 4 * esz);
  rc = in_dtype == S6_BF16 ? launch_bwd_in<uint16_t>(ba, p, vec, st) : launch_bwd_in<float>(ba, p, vec, st);
  if (rc) return rc;
  return in_dtype == S6_BF16 ? launch_sums<uint16_t>(ba, p, dA, dD, ddelta_bias, st)
                             : launch_sums<float>(ba, p, dA, dD, ddelta_bias, st);
}

}  // extern "C"
