// gated.hip -- the gated linear recurrence (include/s6_gated.h): whole
// sequences, gradients and the single-token step.
//
// Per channel, with r = sigmoid(ga + ba), i = sigmoid(gx + bx), v = A r,
// a = e^v, b = sqrt(1 - a^2):
//   h_t = a_t h_{t-1} + u_t,  u_t = b_t i_t x_t
//   lam_t = dy_t + mu_{t+1},  mu_t = a_t lam_t       (adjoint of h_t, backwards)
//   dv = lam (a h_{t-1} - (a^2 / b) i x),  dga = dv A r (1 - r)
//   dx = lam b i,  dgx = lam b x i (1 - i),  dA = sum dv r,  1 - r as e^-z r (z = ga + ba)
// Both recurrences are runs of maps h -> P h + H, which compose, so a tile of
// 128 tokens x 64 channels is reduced to one (P, H) per channel without
// knowing the state that enters it.
//
// One pass: a workgroup loads its tile into registers once, publishes the
// tile's (P, H), takes the state entering the tile from the tiles before it (look_back)
// and writes the tile's outputs.  Inputs are read once and outputs written once,
// at any number of rows and any length.  Workgroups draw their tiles in order
// from a counter, so the tiles that one waits for belong to workgroups that
// run already: every wait ends.  The state entering tile k is always formed as
// P_{k-1} s_{k-1} + H_{k-1}, whichever of these a workgroup reads or forms
// itself, so repeated calls give identical bits.
//
// (A single-pass prefix scan with decoupled look-back, a published method.)
//
// Measured (bf16, us; floor: the bytes of one pass at 6.25 TB/s, what a large
// elementwise pass reaches): 8 x 2048 tokens of 5120 channels 137 (floor 107; 4.9
// TB/s), 65536 tokens of 1536 183 (129), 2 x 2048 of 1536 18 (8), the gradients of
// 8 x 2048 x 5120 301 (188; 3.9 TB/s).  Neither HBM nor the VALU is full: 35
// instructions an element, six of them transcendental, take 71 % of the busy cycles
// (gradients 92 and 76 %); loads, walk and stores of a workgroup follow one
// another.  Passes that first reduce segments and then read all inputs again would
// take 1.75 times the bytes.
#include "s6_gated.h"

#include "block_internal.h"

namespace s6i {

namespace {

constexpr int kGC = 64;                // channels of a tile
constexpr int kGT = S6_GATED_TOKENS;   // tokens of a tile
constexpr int64_t kMaxRow = 1 << 24;   // most elements from token to token
constexpr int kMaxTiles = 1 << 22; // workgroups of a launch (threads below 2^32)
// Waves of a workgroup, and of a SIMD, which the registers leave room for.  The
// forward on pairs of bf16: four of 16 tokens by two channels per lane, 124
// VGPRs (eight of 8 tokens, six per SIMD: 65536 tokens of 1536 187 us, else 183;
// 8 x 2048 of 5120 141, else 137); fp32 would spill there.  Gradients with 16
// waves a workgroup: training of 8 x 2048 x 5120 599 us, with eight 443.
template <typename In, int VEC>
constexpr int kFwdW = sizeof(In) == 2 && VEC == 2 ? 4 : 8;
template <typename In, int VEC>
constexpr int kFwdWaves = kFwdW<In, VEC> == 4 ? 4 : 6;
constexpr int kBwdW = 8, kBwdWaves = 4;
constexpr int kXcds = 8;               // counters of tiles, each in a line of its own
constexpr int kTicketStep = 32;        // words from one to the next

struct GatedArgs {
  const void* x; const void* ga; const void* gx;
  const float* A; const float* ba; const float* bx;
  const uint8_t* starts;
  const float* first;    // h0 (forward), dh_last (backward); nullable
  const float* states;   // backward: the state entering every tile
  float* states_out;     // forward, nullable
  void* y;               // forward, nullable
  float* last;           // h_last (forward), dh0 (backward); nullable
  const void* dy; void* dx; void* dga; void* dgx;
  float* parts;          // column sums' parts (tiles, 3, kGC), nullable
  uint64_t* slots;       // (cols, chunks, kGC), null where a sequence is one tile
  uint32_t* ticket;
  int64_t L;
  int64_t x_batch, x_token, a_batch, a_token, g_batch, g_token;
  int dim;
  int cblocks, cols, chunks, tiles;
  int xcds;              // log2 of the runs of columns, each with a counter
  int base;              // first workgroup of the launch
  int unit;
  int stream;            // outputs' rows are whole lines
  int overlap;           // backward: token rows of an input overlap within a tile
};

// ------------------------------------------------------------- look back --
// A tile's word: {P, H} of the tile, {kState, s} once the state s after the
// tile is known, or kEmpty (both halves written at once).
constexpr uint32_t kEmpty = 0xffffffffu, kState = 0xfffffffeu;
constexpr int kStash = 32;      // tiles whose maps are kept on the way to a known state
constexpr int kMaxPolls = 1 << 21;

__device__ __forceinline__ uint64_t word(uint32_t lo, float h) {
  return (uint64_t)__float_as_uint(h) << 32 | lo;
}
__device__ __forceinline__ uint32_t low(uint64_t w) { return (uint32_t)w; }
__device__ __forceinline__ float high(uint64_t w) { return __uint_as_float((uint32_t)(w >> 32)); }
__device__ __forceinline__ uint64_t peek(const uint64_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void post(uint64_t* p, uint64_t w) {
  __hip_atomic_store(p, w, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// P h + H; a P with its sign set is 0 by a start: nothing of h passes, not
// even a NaN.
__device__ __forceinline__ float pass(float P, float H, float h) {
  return (__float_as_uint(P) >> 31) ? H : __builtin_fmaf(P, h, H);
}

// The state entering tile q > 0 for this lane's channel (whole waves call it).
// slot: the lane's word of this tile; the tile before it is kGC words lower.
// w0: that one's word, as seen some time ago.  Goes back over maps, kept in
// stash, to the first tile whose state is known, and forward from there: one
// tile at a time, since the words compete with the inputs for memory (65536
// tokens of 1536, before the outputs passed the caches: 8 at a time 223 us, 4
// 215, 2 210, 1 208).
__device__ __forceinline__ float look_back(const uint64_t* slot, int q, uint64_t w0, uint64_t (*stash)[kGC]) {
  const int lane = threadIdx.x & 63;
  int done = 0;  // maps in the stash: tiles q - 1 to q - done
  uint64_t w = w0;
  for (int polls = 0; polls < kMaxPolls; ++polls) {
    if (__ballot(low(w) == kState) == ~0ull) {
      float h = high(w);
#pragma unroll 4
      for (int i = done - 1; i >= 0; --i) {
        const uint64_t m = stash[i][lane];
        h = pass(__uint_as_float(low(m)), high(m), h);
      }
      return h;
    }
    // a map in every lane (a tile's word is read while it is written, too): on
    // to the tile before, of which there is one, or with a full stash again
    if (__ballot(low(w) == kEmpty || low(w) == kState) == 0 && done < kStash && done + 1 < q) stash[done++][lane] = w;
    w = peek(slot - (int64_t)(done + 1) * kGC);
  }
  return __builtin_nanf("");  // not reached: see the file's head
}

__device__ __forceinline__ uint32_t publishable(float P) { return P != P ? 0x7fc00000u : __float_as_uint(P); }

// ---------------------------------------------------------------- pieces --
// VEC consecutive channels of a token as loaded.
template <typename In, int VEC>
struct Piece {
  In e[VEC];
  __device__ __forceinline__ void load(const In* p) {
#pragma unroll
    for (int v = 0; v < VEC; ++v) e[v] = p[v];
  }
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, uint32_t off) {
    if constexpr (sizeof(e) == 8) {
      const auto w = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, 0);
      __builtin_memcpy(e, &w, 8);
    } else if constexpr (sizeof(e) == 4) {
      const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0);
      __builtin_memcpy(e, &w, 4);
    } else {
      e[0] = __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    }
  }
  __device__ __forceinline__ float get(int v) const { return to_f32(e[v]); }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int v = 0; v < VEC; ++v) e[v] = 0;
  }
  // What is formed from the values before is formed again after this, instead
  // of being kept in registers.
  __device__ __forceinline__ void again() {
    if constexpr (sizeof(e) == 8) {
      uint64_t w;
      __builtin_memcpy(&w, e, 8);
      asm volatile("" : "+v"(w));
      __builtin_memcpy(e, &w, 8);
    } else if constexpr (sizeof(e) == 4) {
      uint32_t w;
      __builtin_memcpy(&w, e, 4);
      asm volatile("" : "+v"(w));
      __builtin_memcpy(e, &w, 4);
    } else {
      asm volatile("" : "+v"(e[0]));
    }
  }
};
// VEC channels of a token, rounded to In.  AUX: 2 for a streaming store.
template <typename In, int VEC, int AUX>
__device__ __forceinline__ void put_as(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&f)[VEC]) {
  typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
  if constexpr (VEC == 2 && sizeof(In) == 4)
    __builtin_amdgcn_raw_buffer_store_b64(u32x2{__float_as_uint(f[0]), __float_as_uint(f[1])}, r, off, 0, AUX);
  else if constexpr (VEC == 2)
    __builtin_amdgcn_raw_buffer_store_b32(bf_pack(f[0], f[1]), r, off, 0, AUX);
  else if constexpr (sizeof(In) == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[0]), r, off, 0, AUX);
  else
    __builtin_amdgcn_raw_buffer_store_b16(from_f32<In>(f[0]), r, off, 0, AUX);
}
// Whole lines are stored past the caches, which the inputs need (8 x 2048 x 5120:
// 143 -> 137 us, training 459 -> 443); lines that two columns share wait there
// for one another (8 x 2048 x 5000 past the caches as well: 159 -> 184 us).
template <typename In, int VEC>
__device__ __forceinline__ void put(__amdgpu_buffer_rsrc_t r, uint32_t off, const float (&f)[VEC], int stream) {
  if (VEC == 2 && stream)
    put_as<In, VEC, 2>(r, off, f);
  else
    put_as<In, VEC, 0>(r, off, f);
}

// sigmoid(g + bias); the sum first, which leaves nothing of either where they cancel.
__device__ __forceinline__ float gate_f(float g, float bias) {
  return fast_rcp(1.0f + fast_exp2((g + bias) * -kLog2e));
}

// A gate in one register, for the gradients, which take r and 1 - r, each to its
// own accuracy near 0: r below one half, else -(1 - r), as e r with e = e^{-(g +
// bias)}.  1 - r from r would keep nothing of an open gate (at g + bias = 12 it is 1 %
// off, from 17 on 0).  The 2^-149 keeps its sign where it is 0.
__device__ __forceinline__ float split_gate(float g, float bias, float& r) {
  const float e = fast_exp2((g + bias) * -kLog2e);
  r = fast_rcp(1.0f + e);
  return r < 0.5f ? r : -__builtin_fmaf(e, r, 0x1p-149f);
}
__device__ __forceinline__ float whole_gate(float s) { return __builtin_amdgcn_fractf(s); }  // r, at most 1 - 2^-24
__device__ __forceinline__ float gate_slope(float s) {  // r (1 - r)
  const float m = __builtin_fabsf(s);
  return __builtin_fmaf(-m, m, m);
}

// 1 - e^{2 v} for v = v2 ln 2 <= 0 and a = e^v: by its series where e^{2v} is
// near 1 (|2 v| < 0.18, five terms, next one 2.6e-7 of the sum), else from a
// (a's rounding there is at most 7e-7 of the difference).
__device__ __forceinline__ float one_less_square(float v2, float a) {
  constexpr float k = 2.0f * kLn2;
  float s = __builtin_fmaf(v2, k * k * k * k * k / 120.0f, k * k * k * k / 24.0f);
  s = __builtin_fmaf(v2, s, k * k * k / 6.0f);
  s = __builtin_fmaf(v2, s, k * k / 2.0f);
  s = __builtin_fmaf(v2, s, k);
  return v2 > -0.13f ? -v2 * s : __builtin_fmaf(-a, a, 1.0f);
}

// Where a lane's tokens lie: W * VEC groups of T tokens, VEC groups to a
// wave (64 / VEC lanes of VEC channels each).  Tiles and columns of tiles are
// counted in 32 bits (the host sees to it).
template <int VEC, int W>
struct Place {
  static constexpr int G = W * VEC, T = kGT / G;
  int group, half, cl, nt;  // half: the group in its wave; nt: tokens of the group that exist
  int col, q, k, b, c0;     // c0: first channel of the tile
  int64_t w0;               // first token of the wave
  bool on;                  // the lane's channels exist
};
template <int VEC, int W, bool BACK>
__device__ __forceinline__ Place<VEC, W> place_of(const GatedArgs& a, int tile) {
  using P = Place<VEC, W>;
  P p;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  p.half = VEC == 2 ? lane >> 5 : 0;
  p.cl = (VEC == 2 ? lane & 31 : lane) * VEC;
  p.group = wave * VEC + p.half;
  p.q = tile / a.cols;
  p.col = tile - p.q * a.cols;
  p.k = BACK ? a.chunks - 1 - p.q : p.q;
  p.b = p.col / a.cblocks;
  p.c0 = (p.col - p.b * a.cblocks) * kGC;
  p.on = p.c0 + p.cl < a.dim;
  p.w0 = (int64_t)p.k * kGT + wave * (VEC * P::T);
  const int64_t left = a.L - p.w0 - p.half * P::T;
  p.nt = left < 0 ? 0 : left < P::T ? (int)left : P::T;
  return p;
}

// The tile of this workgroup, or a.tiles: it has none.  Workgroups go to the
// eight XCDs in turn, and each XCD takes a run of neighbouring columns (of tiles
// along a sequence), since rows that do not begin at a line's start have lines
// that two columns share.  A tile and those before it come from one counter, in
// order.  One run and one counter for all: 2 x 2048 x 1536 25.9 us, else 18.0;
// 8 x 2048 x 5120 154, else 137; training of 8 x 2048 x 5000 522, else 466.
__device__ __forceinline__ int draw_tile(const GatedArgs& a, uint32_t* shared) {
  const int wg = a.base + (int)blockIdx.x;
  const int x = wg & ((1 << a.xcds) - 1);
  const int lo = (int)((int64_t)a.cols * x >> a.xcds), mine = (int)((int64_t)a.cols * (x + 1) >> a.xcds) - lo;
  int t = wg >> a.xcds;
  if (a.slots) {
    if (threadIdx.x == 0) *shared = atomicAdd(a.ticket + x * kTicketStep, 1u);
    __syncthreads();
    t = __builtin_amdgcn_readfirstlane((int)*shared);
  }
  if (t >= mine * a.chunks) return a.tiles;
  const int q = t / mine;
  return q * a.cols + lo + (t - q * mine);
}

// A wave's part of one tensor as a buffer: its tokens of the tile's channels.
// Offsets are the lanes' own: a scalar offset need not be bounds-checked.
// Past its end loads return 0 and stores are dropped, so that tiles need no
// branches at the end of a sequence; a lane past dim may load what lies beside
// the row, and stores nothing.  A tensor that is not given is an empty buffer:
// without gate_x the gate is 0 with a bias of infinity, which makes i = 1.
struct Rows {
  __amdgpu_buffer_rsrc_t buf;
  uint32_t lane, step;  // bytes: of the lane's first piece, from token to token
};
template <typename In, int VEC, int W>
__device__ __forceinline__ Rows rows_of(const void* base, int64_t batch_stride, int64_t token_stride, const GatedArgs& a,
                                        const Place<VEC, W>& p) {
  constexpr int n = VEC * Place<VEC, W>::T;
  // offsets past the rows' end pass the buffer's and do not wrap
  static_assert((uint64_t)(n + 1) * kMaxRow * sizeof(In) < 1ull << 32, "a wave's tokens lie within 32 bits");
  const int64_t left = a.L - p.w0;
  const uint32_t rows = left < 0 || !base ? 0 : left < n ? (uint32_t)left : n;
  const uint32_t cols = a.dim - p.c0 < kGC ? (uint32_t)(a.dim - p.c0) : kGC;
  const uint64_t u = reinterpret_cast<uint64_t>(static_cast<const In*>(base) + p.b * batch_stride + p.w0 * token_stride + p.c0);
  const uint64_t at = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)(u >> 32)) << 32 |
                      (uint32_t)__builtin_amdgcn_readfirstlane((uint32_t)u);
  Rows r;
  r.step = (uint32_t)token_stride * (uint32_t)sizeof(In);
  r.buf = __builtin_amdgcn_make_buffer_rsrc(
      reinterpret_cast<void*>(at), 0,
      __builtin_amdgcn_readfirstlane(rows > 0 ? (rows - 1) * r.step + cols * (uint32_t)sizeof(In) : 0u), 0x00027000);
  r.lane = p.half * (Place<VEC, W>::T * r.step) + p.cl * (uint32_t)sizeof(In);
  return r;
}
template <typename In, int VEC, int T>
__device__ __forceinline__ void load_rows(Piece<In, VEC> (&o)[T], const Rows& r) {
#pragma unroll
  for (int t = 0; t < T; ++t) o[t].load(r.buf, r.lane + t * r.step);
}

// Bit t: token t of the lane's group starts a sequence.
template <int VEC, int W>
__device__ __forceinline__ uint32_t starts_of(const GatedArgs& a, const Place<VEC, W>& p) {
  constexpr int T = Place<VEC, W>::T;
  const int lane = threadIdx.x & 63, t = lane & (T - 1);
  bool st = false;
  if (t < p.nt) st = a.starts[p.b * a.L + p.w0 + p.half * T + t] != 0;
  const uint64_t all = __ballot(st);
  return (uint32_t)(VEC == 2 && lane >= 32 ? all >> 32 : all) & (uint32_t)((1ull << T) - 1);
}

// --------------------------------------------------------------- forward --
template <typename In, int VEC, bool UNIT, bool STARTS>
__global__ __launch_bounds__((kFwdW<In, VEC> * 64), (kFwdWaves<In, VEC>)) void s6_gated_scan_kernel(GatedArgs a) {
  constexpr int W = kFwdW<In, VEC>;
  using P = Place<VEC, W>;
  constexpr int G = P::G, T = P::T;
  __shared__ float2 agg[G][kGC];
  __shared__ float hin[G][kGC];
  __shared__ uint64_t stash[kStash][kGC];
  __shared__ uint32_t drawn;
  const int tile = draw_tile(a, &drawn);
  if (tile >= a.tiles) return;
  const P p = place_of<VEC, W, false>(a, tile);
  uint64_t* const slot = a.slots + ((int64_t)p.col * a.chunks + p.q) * kGC + (threadIdx.x & 63);
  const uint64_t before = p.q > 0 && threadIdx.x < 64 ? peek(slot - kGC) : ~0ull;
  Piece<In, VEC> xr[T], ar[T], gr[T];
  load_rows(ar, rows_of<In>(a.ga, a.a_batch, a.a_token, a, p));
  load_rows(xr, rows_of<In>(a.x, a.x_batch, a.x_token, a, p));
  load_rows(gr, rows_of<In>(a.gx, a.g_batch, a.g_token, a, p));
  uint32_t starts = 0;
  if constexpr (STARTS) starts = starts_of(a, p);
  float A2[VEC], ba[VEC], bx[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const int c = p.on ? p.c0 + p.cl + v : a.dim - 1;
    A2[v] = a.A[c] * kLog2e;
    ba[v] = a.ba ? a.ba[c] : 0.0f;
    bx[v] = !a.gx ? __builtin_inff() : a.bx ? a.bx[c] : 0.0f;
  }
  float av[T][VEC], uv[T][VEC], Pl[VEC], Hl[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) { Pl[v] = 1.0f; Hl[v] = 0.0f; }
  // (tokens past the end make the last tile's map meaningless: nobody reads it)
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const bool st = STARTS && (starts >> t & 1);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      // (at a start v = -infinity: a = 0, b = 1)
      const float v2 = st ? -__builtin_inff() : A2[v] * gate_f(ar[t].get(v), ba[v]);
      const float d = fast_exp2(v2);
      float u = xr[t].get(v) * gate_f(gr[t].get(v), bx[v]);
      if constexpr (!UNIT) u *= __builtin_amdgcn_sqrtf(one_less_square(v2, d));
      av[t][v] = d;
      uv[t][v] = u;
      Pl[v] *= d;
      Hl[v] = st ? u : __builtin_fmaf(d, Hl[v], u);
    }
  }
  if constexpr (STARTS)
#pragma unroll
    for (int v = 0; v < VEC; ++v) Pl[v] = starts ? -0.0f : __builtin_fabsf(Pl[v]);
#pragma unroll
  for (int v = 0; v < VEC; ++v) agg[p.group][p.cl + v] = make_float2(Pl[v], Hl[v]);
  __syncthreads();
  if (threadIdx.x < 64) {  // the first wave: one channel per lane
    const int lane = threadIdx.x, c = p.c0 + lane;
    float Pt = 1.0f, Ht = 0.0f;
#pragma unroll 4
    for (int i = 0; i < G; ++i) {
      const float2 g = agg[i][lane];
      Ht = pass(g.x, g.y, Ht);
      Pt = (STARTS && __float_as_uint(g.x) >> 31) ? g.x : g.x * Pt;
    }
    float h;
    if (p.q == 0) {
      h = a.first && c < a.dim ? a.first[(int64_t)p.b * a.dim + c] : 0.0f;
    } else {
      post(slot, word(publishable(Pt), Ht));
      h = look_back(slot, p.q, before, stash);
    }
    if (p.q + 1 < a.chunks) post(slot, word(kState, pass(Pt, Ht, h)));
    if (a.states_out && c < a.dim) a.states_out[((int64_t)p.b * a.chunks + p.k) * a.dim + c] = h;
#pragma unroll 4
    for (int i = 0; i < G; ++i) {
      const float2 g = agg[i][lane];
      hin[i][lane] = h;
      h = pass(g.x, g.y, h);
    }
  }
  __syncthreads();
  if (!a.y || !p.on) return;
  float h[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) h[v] = hin[p.group][p.cl + v];
  auto next = [&](int t) {
#pragma unroll
    for (int v = 0; v < VEC; ++v)
      h[v] = STARTS && (starts >> t & 1) ? uv[t][v] : __builtin_fmaf(av[t][v], h[v], uv[t][v]);
  };
  if (a.last && p.k + 1 == a.chunks) {  // the state after the last token
#pragma unroll
    for (int t = 0; t < T; ++t) {
      next(t);
      if (p.w0 + p.half * T + t + 1 == a.L) {
#pragma unroll
        for (int v = 0; v < VEC; ++v) a.last[(int64_t)p.b * a.dim + p.c0 + p.cl + v] = h[v];
      }
    }
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = hin[p.group][p.cl + v];
  }
  const Rows y = rows_of<In>(a.y, a.L * a.dim, a.dim, a, p);
#pragma unroll
  for (int t = 0; t < T; ++t) {
    next(t);
    put<In, VEC>(y.buf, y.lane + t * y.step, h, a.stream);
  }
}

// -------------------------------------------------------------- backward --
template <typename In, int VEC, bool UNIT, bool STARTS>
__global__ __launch_bounds__(kBwdW * 64, kBwdWaves) void s6_gated_scan_bwd_kernel(GatedArgs a) {
  using P = Place<VEC, kBwdW>;
  constexpr int G = P::G, T = P::T;
  __shared__ float agg[3][G][kGC];   // P, H, M of the groups; later the column sums
  __shared__ float ent[2][G][kGC];   // the state entering a group, the adjoint leaving it
  __shared__ uint64_t stash[kStash][kGC];
  __shared__ uint32_t drawn;
  const int tile = draw_tile(a, &drawn);
  if (tile >= a.tiles) return;
  const P p = place_of<VEC, kBwdW, true>(a, tile);
  uint64_t* const slot = a.slots + ((int64_t)p.col * a.chunks + p.q) * kGC + (threadIdx.x & 63);
  const uint64_t before = p.q > 0 && threadIdx.x < 64 ? peek(slot - kGC) : ~0ull;
  Piece<In, VEC> xr[T], ar[T], gr[T], yr[T];
  load_rows(ar, rows_of<In>(a.ga, a.a_batch, a.a_token, a, p));
  load_rows(xr, rows_of<In>(a.x, a.x_batch, a.x_token, a, p));
  load_rows(gr, rows_of<In>(a.gx, a.g_batch, a.g_token, a, p));
  load_rows(yr, rows_of<In>(a.dy, a.L * a.dim, a.dim, a, p));
  if (a.overlap) {  // (a row past the end then lies in part before the buffer's)
#pragma unroll
    for (int t = 0; t < T; ++t)
      if (t >= p.nt) { ar[t].clear(); xr[t].clear(); gr[t].clear(); }
  }
  uint32_t starts = 0;
  if constexpr (STARTS) starts = starts_of(a, p);
  float Ac[VEC], ba[VEC], bx[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const int c = p.on ? p.c0 + p.cl + v : a.dim - 1;
    Ac[v] = a.A[c];
    ba[v] = a.ba ? a.ba[c] : 0.0f;
    bx[v] = !a.gx ? __builtin_inff() : a.bx ? a.bx[c] : 0.0f;
  }
  // the gates, decays and inputs, and the group's maps
  float av[T][VEC], rv[T][VEC], iv[T][VEC], uv[T][VEC], sv[T][VEC];
  float Pl[VEC], Hl[VEC], Ml[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) { Pl[v] = 1.0f; Hl[v] = Ml[v] = 0.0f; }
  // (a token past the end, with a = 1 and dy = 0, hands the adjoint on)
#pragma unroll
  for (int t = 0; t < T; ++t) {
    const bool st = STARTS && (starts >> t & 1);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      float r, i;
      rv[t][v] = split_gate(ar[t].get(v), ba[v], r);
      iv[t][v] = split_gate(gr[t].get(v), bx[v], i);
      if (st) rv[t][v] = 0.0f;  // (a start's gate enters nothing, not as 0 times a NaN either)
      // formed here, not where they are used next with e and r kept until then
      // (training of 8 x 2048 x 5120 586 us, else 445)
      asm volatile("" : "+v"(rv[t][v]), "+v"(iv[t][v]));
      const float v2 = st ? -__builtin_inff() : Ac[v] * kLog2e * r;
      float d = fast_exp2(v2);
      float u = i * xr[t].get(v);
      if constexpr (!UNIT) {
        sv[t][v] = one_less_square(v2, d);
        u *= __builtin_amdgcn_sqrtf(sv[t][v]);
      }
      if (t >= p.nt) d = 1.0f;
      av[t][v] = d;
      uv[t][v] = u;
      Pl[v] *= d;
      Hl[v] = st ? u : __builtin_fmaf(d, Hl[v], u);
    }
  }
  if constexpr (STARTS)
#pragma unroll
    for (int v = 0; v < VEC; ++v) Pl[v] = starts ? -0.0f : __builtin_fabsf(Pl[v]);
#pragma unroll
  for (int t = T - 1; t >= 0; --t) {
    const bool st = STARTS && (starts >> t & 1);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float m = av[t][v] * (yr[t].get(v) + Ml[v]);
      Ml[v] = st ? 0.0f : m;
    }
  }
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    agg[0][p.group][p.cl + v] = Pl[v];
    agg[1][p.group][p.cl + v] = Hl[v];
    agg[2][p.group][p.cl + v] = Ml[v];
  }
  __syncthreads();
  if (threadIdx.x < 64) {
    const int lane = threadIdx.x, c = p.c0 + lane;
    const bool on = c < a.dim;
    float h = on ? a.states[((int64_t)p.b * a.chunks + p.k) * a.dim + c] : 0.0f;
    float Pt = 1.0f, Mt = 0.0f;
#pragma unroll 4
    for (int i = 0; i < G; ++i) {
      ent[0][i][lane] = h;
      h = pass(agg[0][i][lane], agg[1][i][lane], h);
    }
#pragma unroll 4
    for (int i = G - 1; i >= 0; --i) {
      const float gp = agg[0][i][lane];
      Mt = pass(gp, agg[2][i][lane], Mt);
      Pt = (STARTS && __float_as_uint(gp) >> 31) ? gp : gp * Pt;
    }
    float m;
    if (p.q == 0) {
      m = a.first && on ? a.first[(int64_t)p.b * a.dim + c] : 0.0f;
    } else {
      post(slot, word(publishable(Pt), Mt));
      m = look_back(slot, p.q, before, stash);
    }
    if (p.q + 1 < a.chunks) post(slot, word(kState, pass(Pt, Mt, m)));
#pragma unroll 4
    for (int i = G - 1; i >= 0; --i) {
      ent[1][i][lane] = m;
      m = pass(agg[0][i][lane], agg[2][i][lane], m);
    }
    if (a.last && p.q + 1 == a.chunks && on) a.last[(int64_t)p.b * a.dim + c] = m;
  }
  __syncthreads();
  // The state before each token (in place of the inputs), then backwards with
  // the adjoint.
  float h[VEC], m[VEC], sA[VEC], sa[VEC], sx[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    h[v] = ent[0][p.group][p.cl + v];
    m[v] = ent[1][p.group][p.cl + v];
    sA[v] = sa[v] = sx[v] = 0.0f;
  }
#pragma unroll
  for (int t = 0; t < T; ++t) {
    xr[t].again();
    yr[t].again();
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      const float u = uv[t][v];
      uv[t][v] = t < p.nt ? h[v] : 0.0f;  // (a last state that is infinite goes no further)
      h[v] = STARTS && (starts >> t & 1) ? u : __builtin_fmaf(av[t][v], h[v], u);
    }
  }
  const Rows dx = rows_of<In>(a.dx, a.L * a.dim, a.dim, a, p);
  const Rows dga = rows_of<In>(a.dga, a.L * a.dim, a.dim, a, p);
  const Rows dgx = rows_of<In>(a.dgx, a.L * a.dim, a.dim, a, p);
  if (p.on) {
#pragma unroll
    for (int t = T - 1; t >= 0; --t) {
      const bool st = STARTS && (starts >> t & 1), none = t >= p.nt;
      float ox[VEC], oa[VEC], og[VEC];
#pragma unroll
      for (int v = 0; v < VEC; ++v) {
        const float x = xr[t].get(v), d = av[t][v], r = whole_gate(rv[t][v]), i = whole_gate(iv[t][v]);
        float lam = yr[t].get(v) + m[v];
        m[v] = st ? 0.0f : d * lam;
        lam = none ? 0.0f : lam;
        float w = d * uv[t][v], lb = lam;  // lb: lam b
        if constexpr (!UNIT) {
          const float s = sv[t][v];
          const float inv = s >= 0x1p-126f ? __builtin_amdgcn_rsqf(s) : 0.0f;  // 1 / b
          w = __builtin_fmaf(-d * d * inv, i * x, w);
          lb *= s * inv;
        }
        const float dv = st ? 0.0f : lam * w;
        ox[v] = lb * i;
        oa[v] = dv * (Ac[v] * gate_slope(rv[t][v]));
        og[v] = lb * x * gate_slope(iv[t][v]);
        sA[v] = __builtin_fmaf(dv, r, sA[v]);
        sa[v] += oa[v];
        sx[v] += og[v];
      }
      put<In, VEC>(dx.buf, dx.lane + t * dx.step, ox, a.stream);
      put<In, VEC>(dga.buf, dga.lane + t * dga.step, oa, a.stream);
      put<In, VEC>(dgx.buf, dgx.lane + t * dgx.step, og, a.stream);
    }
  }
  if (!a.parts) return;
  // (the groups' maps were read before the barrier above)
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    agg[0][p.group][p.cl + v] = sA[v];
    agg[1][p.group][p.cl + v] = sa[v];
    agg[2][p.group][p.cl + v] = sx[v];
  }
  __syncthreads();
  if (threadIdx.x < 3 * kGC) {
    const int which = threadIdx.x / kGC, l = threadIdx.x % kGC;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < G; ++i) s += agg[which][i][l];
    a.parts[(((int64_t)p.col * a.chunks + p.k) * 3 + which) * kGC + l] = s;
  }
}

// Sums of the parts over rows and chunks.  blockIdx.x: block of 64 channels;
// blockIdx.y: which sum; blockIdx.z: a slice of the parts.
// part (n, 3, kGC) of channel block cb: index (b * cblocks + cb) * chunks + k.
struct SumArgs {
  const float* parts;
  float* out[3];       // nullable
  float* slices;       // (slices, cblocks, 3, kGC) where there are several
  int64_t batch, chunks, cblocks, dim, per;  // per: parts of a slice
};
__global__ __launch_bounds__(512) void s6_gated_colsum_kernel(SumArgs a) {
  __shared__ float buf[8][kGC];
  const int which = blockIdx.y, l = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int64_t n = a.batch * a.chunks, cb = blockIdx.x;
  const int64_t lo = blockIdx.z * a.per, hi = lo + a.per < n ? lo + a.per : n;
  float s = 0.0f;
#pragma unroll 4
  for (int64_t i = lo + w; i < hi; i += 8) {
    const int64_t b = i / a.chunks, k = i - b * a.chunks;
    s += a.parts[(((b * a.cblocks + cb) * a.chunks + k) * 3 + which) * kGC + l];
  }
  buf[w][l] = s;
  __syncthreads();
  if (w) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += buf[i][l];
  const int64_t c = cb * kGC + l;
  if (a.slices)
    a.slices[((blockIdx.z * a.cblocks + cb) * 3 + which) * kGC + l] = s;
  else if (a.out[which] && c < a.dim)
    a.out[which][c] = s;
}
__global__ __launch_bounds__(64) void s6_gated_slices_kernel(SumArgs a, int64_t slices) {
  const int which = blockIdx.y, l = threadIdx.x;
  const int64_t cb = blockIdx.x, c = cb * kGC + l;
  float s = 0.0f;
#pragma unroll 4
  for (int64_t i = 0; i < slices; ++i) s += a.slices[((i * a.cblocks + cb) * 3 + which) * kGC + l];
  if (a.out[which] && c < a.dim) a.out[which][c] = s;
}

// Counters at 0 and empty words, two of them per store.
__global__ __launch_bounds__(256) void s6_gated_init_kernel(u32x4* slots, int64_t pairs, uint32_t* ticket) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i < kXcds) ticket[i * kTicketStep] = 0;
  if (i < pairs) slots[i] = u32x4{kEmpty, kEmpty, kEmpty, kEmpty};
}

// ------------------------------------------------------------------ step --
// A channel to a lane, or two.  256 x 5120: 6.0 us (floor 3.4: 21 MB), one row of
// 1536 2.5, the launch.
template <typename In, int VEC>
__global__ __launch_bounds__(256) void s6_gated_step_kernel(GatedArgs a, float* hs) {
  const int64_t per = (a.dim + VEC - 1) / VEC, i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t b = (int64_t)a.base + blockIdx.y;
  const int64_t c = i0 * VEC;
  if (i0 >= per) return;
  Piece<In, VEC> xr, ar, gr;
  xr.load(static_cast<const In*>(a.x) + b * a.x_batch + c);
  ar.load(static_cast<const In*>(a.ga) + b * a.a_batch + c);
  if (a.gx) gr.load(static_cast<const In*>(a.gx) + b * a.g_batch + c);
  Piece<float, VEC> hr;
  hr.load(hs + b * a.dim + c);
  float h[VEC];
#pragma unroll
  for (int v = 0; v < VEC; ++v) {
    const float v2 = a.A[c + v] * kLog2e * gate_f(ar.get(v), a.ba ? a.ba[c + v] : 0.0f);
    const float d = fast_exp2(v2);
    float u = xr.get(v);
    if (a.gx) u *= gate_f(gr.get(v), a.bx ? a.bx[c + v] : 0.0f);
    if (!a.unit) u *= __builtin_amdgcn_sqrtf(one_less_square(v2, d));
    h[v] = __builtin_fmaf(d, hr.get(v), u);
  }
  In* y = static_cast<In*>(a.y) + b * a.dim + c;
  if constexpr (VEC == 2) {
    *reinterpret_cast<float2*>(hs + b * a.dim + c) = make_float2(h[0], h[1]);
    if constexpr (sizeof(In) == 2) *reinterpret_cast<uint32_t*>(y) = bf_pack(h[0], h[1]);
    else *reinterpret_cast<float2*>(y) = make_float2(h[0], h[1]);
  } else {
    hs[b * a.dim + c] = h[0];
    *y = from_f32<In>(h[0]);
  }
}

// ------------------------------------------------------------------ host --
int check_gated(const s6_gated_dims* d, int in_dtype, int flags, bool gx, bool tokens) {
  if (!d) return S6_ERR_NULL;
  if (in_dtype != S6_F32 && in_dtype != S6_BF16) return S6_ERR_DTYPE;
  if (flags & ~S6_UNIT_INPUT) return S6_ERR_FLAGS;
  if (d->batch < 0 || d->dim < 0 || (tokens && d->seqlen < 0)) return S6_ERR_SHAPE;
  if (d->batch == 0 || d->dim == 0) return S6_OK;
  const int64_t len = tokens && d->seqlen > 0 ? d->seqlen : 1;
  // element counts with headroom for padded tiles and byte sizes
  int64_t t;
  if (d->dim > kMaxRow || d->batch > INT32_MAX || !mul_ok(d->batch, d->dim, &t) || !mul_ok(t, 64 * 16, &t) ||
      !mul_ok(t, len + kGT, &t))
    return S6_ERR_SHAPE;
  // tiles and workgroups in 32 bits, those without a tile included
  const int64_t cols = d->batch * ((d->dim + kGC - 1) / kGC);
  if (!mul_ok(cols + cols / 8 + kXcds, (len + kGT - 1) / kGT, &t) || t > INT32_MAX - kMaxTiles)
    return S6_ERR_SHAPE;
  const int64_t str[] = {d->x_batch, d->x_token, d->a_batch, d->a_token, d->g_batch, d->g_token};
  for (int i = 0; i < (gx ? 6 : 4); ++i) {
    if ((i & 1) && !tokens) continue;
    if (str[i] < 0 || ((i & 1) && len > 1 && str[i] > kMaxRow)) return S6_ERR_SHAPE;
    if (!mul_ok(str[i], (i & 1) ? len : d->batch, &t) || !mul_ok(t, 16, &t)) return S6_ERR_SHAPE;
  }
  return S6_OK;
}

struct GatedWs {
  int64_t cblocks, cols, chunks, tiles, slices, per;
  size_t slots, states, parts, sums, total;  // byte offsets; the counters lie at 0
};
GatedWs gated_ws(const s6_gated_dims& d, bool back, bool has_states) {
  GatedWs w;
  w.cblocks = (d.dim + kGC - 1) / kGC;
  w.cols = d.batch * w.cblocks;
  w.chunks = (d.seqlen + kGT - 1) / kGT;
  w.tiles = w.cols * w.chunks;
  const int64_t n = d.batch * w.chunks;
  // column sums: slices of at least 256 parts, at most 64
  w.slices = n / 256 < 1 ? 1 : n / 256 > 64 ? 64 : n / 256;
  w.per = (n + w.slices - 1) / w.slices;
  w.slots = kXcds * kTicketStep * sizeof(uint32_t);
  size_t at = w.chunks > 1 ? w.slots + (size_t)w.tiles * kGC * sizeof(uint64_t) : 0;
  w.states = w.parts = w.sums = 0;
  if (back) {
    w.states = up256(at);
    at = w.states + (has_states ? 0 : (size_t)n * d.dim * sizeof(float));
    w.parts = up256(at);
    at = w.parts + (size_t)w.tiles * 3 * kGC * sizeof(float);
    w.sums = up256(at);
    at = w.sums + (w.slices > 1 ? (size_t)w.slices * w.cblocks * 3 * kGC * sizeof(float) : 0);
  }
  w.total = up256(at);
  return w;
}

template <typename In, int VEC>
int launch_gated(GatedArgs a, bool back, hipStream_t st) {
  if (a.slots) {
    // 8 tiles a workgroup
    for (int64_t t = 0; t < a.tiles; t += (int64_t)8 * kMaxTiles) {
      const int64_t n = a.tiles - t < (int64_t)8 * kMaxTiles ? a.tiles - t : (int64_t)8 * kMaxTiles;
      hipLaunchKernelGGL(s6_gated_init_kernel, dim3((unsigned)((n + 7) / 8)), dim3(256), 0, st,
                         reinterpret_cast<u32x4*>(a.slots + t * kGC), n * (kGC / 2), a.ticket);
      S6_HIP(hipGetLastError(), "s6_gated_init_kernel launch");
    }
  }
  // runs of columns for the XCDs, where they come out even; as many workgroups
  // for each as the longest run needs
  const int most = (a.cols + kXcds - 1) / kXcds;
  a.xcds = (int64_t)most * kXcds <= a.cols + a.cols / 8 ? 3 : 0;
  const int wgs = (a.xcds ? most * kXcds : a.cols) * a.chunks;
  for (a.base = 0; a.base < wgs; a.base += kMaxTiles) {
    const dim3 grid((unsigned)(wgs - a.base < kMaxTiles ? wgs - a.base : kMaxTiles)), block(64 * (back ? kBwdW : kFwdW<In, VEC>));
#define S6_GATED_LAUNCH(UNIT, STARTS)                                                              \
  if (back)                                                                                        \
    hipLaunchKernelGGL((s6_gated_scan_bwd_kernel<In, VEC, UNIT, STARTS>), grid, block, 0, st, a);  \
  else                                                                                             \
    hipLaunchKernelGGL((s6_gated_scan_kernel<In, VEC, UNIT, STARTS>), grid, block, 0, st, a);
    if (a.unit && a.starts) { S6_GATED_LAUNCH(true, true) }
    else if (a.unit) { S6_GATED_LAUNCH(true, false) }
    else if (a.starts) { S6_GATED_LAUNCH(false, true) }
    else { S6_GATED_LAUNCH(false, false) }
#undef S6_GATED_LAUNCH
    S6_HIP(hipGetLastError(), "s6_gated_scan kernel launch");
  }
  return S6_OK;
}
template <typename In>
int launch_gated_in(const GatedArgs& a, bool back, bool vec, hipStream_t st) {
  return vec ? launch_gated<In, 2>(a, back, st) : launch_gated<In, 1>(a, back, st);
}

GatedArgs gated_args(const s6_gated_dims& d, int flags, const void* x, const void* ga, const float* ba, const void* gx,
                     const float* bx, const float* A) {
  GatedArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x; a.ga = ga; a.gx = gx; a.A = A; a.ba = ba; a.bx = bx;
  a.L = d.seqlen; a.dim = (int)d.dim;
  a.x_batch = d.x_batch; a.a_batch = d.a_batch; a.g_batch = d.g_batch;
  // (a stride along a single token may be anything)
  const bool one = d.seqlen == 1;
  a.x_token = one ? d.dim : d.x_token; a.a_token = one ? d.dim : d.a_token; a.g_token = one ? d.dim : d.g_token;
  a.unit = (flags & S6_UNIT_INPUT) != 0;
  return a;
}

// Rows of outputs are whole lines.
int lines_ok(const s6_gated_dims& d, size_t esz, const void* const* ptrs, int n) {
  bool ok = d.dim * (int64_t)esz % 128 == 0;
  for (int i = 0; i < n; ++i) ok = ok && aligned(ptrs[i], 128);
  return ok;
}

// Token rows of an input that are closer than a tile's columns are wide.
int rows_overlap(const s6_gated_dims& d, bool gx) {
  const int64_t cols = d.dim < kGC ? d.dim : kGC;
  return d.seqlen > 1 && (d.x_token < cols || d.a_token < cols || (gx && d.g_token < cols));
}

// Two channels per lane: every row begins at a multiple of two elements.
bool pairs_ok(const s6_gated_dims& d, bool gx, bool tokens, size_t esz, const void* const* ptrs, int n) {
  bool ok = d.dim % 2 == 0 && d.x_batch % 2 == 0 && d.a_batch % 2 == 0 && (!gx || d.g_batch % 2 == 0);
  if (tokens) ok = ok && d.x_token % 2 == 0 && d.a_token % 2 == 0 && (!gx || d.g_token % 2 == 0);
  for (int i = 0; i < n; ++i) ok = ok && aligned(ptrs[i], 2 * esz);
  return ok;
}

int check_ptrs(const void* const* ins, int n, size_t esz, const void* const* f32s, int m) {
  for (int i = 0; i < n; ++i)
    if (!aligned(ins[i], esz)) return S6_ERR_ALIGN;
  for (int i = 0; i < m; ++i)
    if (!aligned(f32s[i], 4)) return S6_ERR_ALIGN;
  return S6_OK;
}

}  // namespace

}  // namespace s6i

using namespace s6i;

extern "C" {

int s6_gated_scan_fwd_workspace_size(const s6_gated_dims* d, size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  const int rc = check_gated(d, S6_F32, 0, true, true);
  if (rc) return rc;
  *bytes = d->batch == 0 || d->dim == 0 || d->seqlen == 0 ? 0 : gated_ws(*d, false, true).total;
  return S6_OK;
}

int s6_gated_scan_fwd(const s6_gated_dims* d, int in_dtype, int flags, const void* x, const void* gate_a,
                      const float* bias_a, const void* gate_x, const float* bias_x, const float* A,
                      const uint8_t* starts, const float* h0, void* y, float* h_last, float* states, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int rc = check_gated(d, in_dtype, flags, gate_x != nullptr, true);
  if (rc) return rc;
  if (d->batch == 0 || d->dim == 0) return S6_OK;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4;
  if (d->seqlen > 0 && (!x || !gate_a || !A || !y || (bias_x && !gate_x))) return S6_ERR_NULL;
  const void* ins[] = {x, gate_a, gate_x, y};
  const void* f32s[] = {bias_a, bias_x, A, h0, h_last, states};
  if ((rc = check_ptrs(ins, 4, esz, f32s, 6))) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (d->seqlen == 0) return h_last ? launch_copy_state(h0, h_last, d->batch * d->dim, st) : S6_OK;
  const GatedWs w = gated_ws(*d, false, true);
  if (w.total > 0) {
    if (!workspace || workspace_bytes < w.total) return S6_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return S6_ERR_ALIGN;
  }
  GatedArgs a = gated_args(*d, flags, x, gate_a, bias_a, gate_x, bias_x, A);
  a.starts = starts; a.first = h0; a.states_out = states; a.y = y; a.last = h_last;
  a.cblocks = (int)w.cblocks; a.cols = (int)w.cols; a.chunks = (int)w.chunks; a.tiles = (int)w.tiles;
  if (w.chunks > 1) {
    a.ticket = static_cast<uint32_t*>(workspace);
    a.slots = reinterpret_cast<uint64_t*>(static_cast<char*>(workspace) + w.slots);
  }
  a.stream = lines_ok(*d, esz, ins + 3, 1);
  const bool vec = pairs_ok(*d, gate_x != nullptr, true, esz, ins, 4);
  return in_dtype == S6_BF16 ? launch_gated_in<uint16_t>(a, false, vec, st) : launch_gated_in<float>(a, false, vec, st);
}

int s6_gated_scan_bwd_workspace_size(const s6_gated_dims* d, int has_states, size_t* bytes) {
  if (!bytes) return S6_ERR_NULL;
  const int rc = check_gated(d, S6_F32, 0, true, true);
  if (rc) return rc;
  *bytes = d->batch == 0 || d->dim == 0 || d->seqlen == 0 ? 0 : gated_ws(*d, true, has_states != 0).total;
  return S6_OK;
}

int s6_gated_scan_bwd(const s6_gated_dims* d, int in_dtype, int flags, const void* x, const void* gate_a,
                      const float* bias_a, const void* gate_x, const float* bias_x, const float* A,
                      const uint8_t* starts, const float* h0, const float* states, const void* dy,
                      const float* dh_last, void* dx, void* dgate_a, void* dgate_x, float* dA, float* dbias_a,
                      float* dbias_x, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_gated(d, in_dtype, flags, gate_x != nullptr, true);
  if (rc) return rc;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4;
  const bool work = d->batch > 0 && d->dim > 0 && d->seqlen > 0;
  if (work && (!x || !gate_a || !A || !dy || !dx || !dgate_a || (gate_x && !dgate_x) ||
               ((bias_x || dbias_x || dgate_x) && !gate_x)))
    return S6_ERR_NULL;
  const void* ins[] = {x, gate_a, gate_x, dy, dx, dgate_a, dgate_x};
  const void* f32s[] = {bias_a, bias_x, A, h0, states, dh_last, dA, dbias_a, dbias_x, dh0};
  if ((rc = check_ptrs(ins, 7, esz, f32s, 10))) return rc;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (!work) {  // sums of nothing
    fill(dA, 0.0f, d->dim, st);
    fill(dbias_a, 0.0f, d->dim, st);
    fill(dbias_x, 0.0f, d->dim, st);
    if ((dA || dbias_a || dbias_x) && d->dim > 0) S6_HIP(hipGetLastError(), "s6_fill launch");
    return dh0 && d->batch * d->dim > 0 ? launch_copy_state(dh_last, dh0, d->batch * d->dim, st) : S6_OK;
  }
  const GatedWs w = gated_ws(*d, true, states != nullptr);
  if (!workspace || workspace_bytes < w.total) return S6_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return S6_ERR_ALIGN;
  char* ws = static_cast<char*>(workspace);
  GatedArgs a = gated_args(*d, flags, x, gate_a, bias_a, gate_x, bias_x, A);
  a.starts = starts;
  a.cblocks = (int)w.cblocks; a.cols = (int)w.cols; a.chunks = (int)w.chunks; a.tiles = (int)w.tiles;
  if (w.chunks > 1) {
    a.ticket = reinterpret_cast<uint32_t*>(ws);
    a.slots = reinterpret_cast<uint64_t*>(ws + w.slots);
  }
  a.stream = lines_ok(*d, esz, ins + 4, 3);
  const bool vec = pairs_ok(*d, gate_x != nullptr, true, esz, ins, 7);
  const auto launch = [&](bool back) {
    return in_dtype == S6_BF16 ? launch_gated_in<uint16_t>(a, back, vec, st) : launch_gated_in<float>(a, back, vec, st);
  };
  if (!states) {  // the forward without y
    a.first = h0;
    a.states_out = reinterpret_cast<float*>(ws + w.states);
    if ((rc = launch(false))) return rc;
    a.states_out = nullptr;
    states = reinterpret_cast<float*>(ws + w.states);
  }
  a.states = states; a.first = dh_last; a.last = dh0;
  a.overlap = rows_overlap(*d, gate_x != nullptr);
  a.dy = dy; a.dx = dx; a.dga = dgate_a; a.dgx = dgate_x;
  const bool sums = dA || dbias_a || dbias_x;
  a.parts = sums ? reinterpret_cast<float*>(ws + w.parts) : nullptr;
  if ((rc = launch(true))) return rc;
  if (!sums) return S6_OK;
  SumArgs s;
  s.parts = a.parts;
  s.out[0] = dA; s.out[1] = dbias_a; s.out[2] = dbias_x;
  s.slices = w.slices > 1 ? reinterpret_cast<float*>(ws + w.sums) : nullptr;
  s.batch = d->batch; s.chunks = w.chunks; s.cblocks = w.cblocks; s.dim = d->dim; s.per = w.per;
  hipLaunchKernelGGL(s6_gated_colsum_kernel, dim3((unsigned)w.cblocks, 3, (unsigned)w.slices), dim3(512), 0, st, s);
  S6_HIP(hipGetLastError(), "s6_gated_colsum_kernel launch");
  if (w.slices > 1) {
    hipLaunchKernelGGL(s6_gated_slices_kernel, dim3((unsigned)w.cblocks, 3), dim3(64), 0, st, s, w.slices);
    S6_HIP(hipGetLastError(), "s6_gated_slices_kernel launch");
  }
  return S6_OK;
}

int s6_gated_state_update(const s6_gated_dims* d, int in_dtype, int flags, float* h, const void* x,
                          const void* gate_a, const float* bias_a, const void* gate_x, const float* bias_x,
                          const float* A, void* y, void* stream) {
  int rc = check_gated(d, in_dtype, flags, gate_x != nullptr, false);
  if (rc) return rc;
  if (d->batch == 0 || d->dim == 0) return S6_OK;
  if (!h || !x || !gate_a || !A || !y || (bias_x && !gate_x)) return S6_ERR_NULL;
  const size_t esz = in_dtype == S6_BF16 ? 2 : 4;
  const void* ins[] = {x, gate_a, gate_x, y};
  const void* f32s[] = {h, bias_a, bias_x, A};
  if ((rc = check_ptrs(ins, 4, esz, f32s, 4))) return rc;
  GatedArgs a = gated_args(*d, flags, x, gate_a, bias_a, gate_x, bias_x, A);
  a.y = y;
  const bool vec = pairs_ok(*d, gate_x != nullptr, false, esz, ins, 4) && aligned(h, 8);
  hipStream_t st = static_cast<hipStream_t>(stream);
  const int64_t per = vec ? (d->dim + 1) / 2 : d->dim;
  for (int64_t b0 = 0; b0 < d->batch; b0 += 65535) {
    a.base = (int)b0;
    const int64_t rows = d->batch - b0 < 65535 ? d->batch - b0 : 65535;
    const dim3 grid((unsigned)((per + 255) / 256), (unsigned)rows);
    if (in_dtype == S6_BF16) {
      if (vec) hipLaunchKernelGGL((s6_gated_step_kernel<uint16_t, 2>), grid, dim3(256), 0, st, a, h);
      else hipLaunchKernelGGL((s6_gated_step_kernel<uint16_t, 1>), grid, dim3(256), 0, st, a, h);
    } else {
      if (vec) hipLaunchKernelGGL((s6_gated_step_kernel<float, 2>), grid, dim3(256), 0, st, a, h);
      else hipLaunchKernelGGL((s6_gated_step_kernel<float, 1>), grid, dim3(256), 0, st, a, h);
    }
    S6_HIP(hipGetLastError(), "s6_gated_step_kernel launch");
  }
  return S6_OK;
}

}  // extern "C"
